"""Rotary positions with several axes and the paged 8-bit cache without a GPU: pins of the oracle's definitions
and the refusals of the C entry points and the binding."""
import ctypes

import numpy as np
import pytest

from oracle import rope_rotate
from oracle.cache8 import append, attention, dense_cache, limits, page_scale, rotate_axes
from oracle.fp8 import e4m3_decode, e4m3_encode
from streaming_causal_video_timestep_b200 import _lib


@pytest.fixture(scope="module")
def lib():
    from streaming_causal_video_timestep_b200 import build
    build.build()
    return _lib.load()


# ---- the oracle ----------------------------------------------------------------------------
def test_rotation_is_the_streams_rope_on_three_axes():
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((9, 2, 64)), rng.integers(-50, 50, (9, 3))
    ref = rope_rotate(x, pos[:, 0], pos[:, 1], pos[:, 2], (12, 10, 10), 10000.0)
    np.testing.assert_allclose(rotate_axes(x, pos, (12, 10, 10)), ref, rtol=0, atol=1e-14)
    # halves: the same pairs, elsewhere in the row
    perm = np.concatenate([np.arange(0, 64, 2), np.arange(1, 64, 2)])
    np.testing.assert_allclose(rotate_axes(x[..., perm], pos, (12, 10, 10), half=True), ref[..., perm], rtol=0, atol=1e-14)


@pytest.mark.parametrize("half", [False, True])
def test_inverse_is_the_gradient(half):
    rng = np.random.default_rng(1)
    x, g, pos = rng.standard_normal((4, 2, 24)), rng.standard_normal((4, 2, 24)), rng.integers(0, 90, (4, 2))
    pairs = (3, 5)                                       # 16 rotated elements, 8 passed through
    dx = rotate_axes(g, pos, pairs, half=half, inverse=True)
    f = lambda y: float((rotate_axes(y, pos, pairs, half=half) * g).sum())  # noqa: E731
    for i in [(0, 0, 0), (1, 1, 5), (2, 0, 15), (3, 1, 16), (3, 1, 23)]:
        e = np.zeros_like(x)
        e[i] = 1e-4
        # linear in x: the central difference is exact up to rounding of two sums of ~200 terms (2e-14) over 2e-4
        assert abs((f(x + e) - f(x - e)) / 2e-4 - dx[i]) < 1e-9
    np.testing.assert_allclose(rotate_axes(dx, pos, pairs, half=half), g, rtol=0, atol=1e-14)


def test_page_scale_is_the_smallest_power_of_two():
    for a in (448.0, np.nextafter(448.0, 500), 1.0, 1e-3, 1.75, 3.5, 3e38, 2.0 ** -140):
        s = page_scale(a)
        assert 448 * s >= a and (s == 2.0 ** -64 or 448 * (s / 2) < a)
    assert page_scale(0.0) == 2.0 ** -64 and np.isnan(page_scale(np.inf)) and np.isnan(page_scale(np.nan))


def test_append_in_pieces_and_growth():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((70, 2, 64)).astype(np.float32)
    x[40:] *= 8.0                                        # page 1 (tokens 32..63) grows at token 40
    table = np.array([[2, 0, 1]])
    one = np.zeros((3, 2, 32, 64), np.uint8), np.ones((3, 2))
    append(x, *one, table, [0], [0, 70])
    two = np.zeros((3, 2, 32, 64), np.uint8), np.ones((3, 2))
    for a, b in ((0, 5), (5, 40), (40, 70)):
        append(x[a:b], *two, table, [a], [0, b - a])
    np.testing.assert_array_equal(one[1], two[1])
    # a code that was written under a smaller scale was rounded twice: within a half step of each rounding
    d1, d2 = (dense_cache(*c, table, 0, 70) for c in (one, two))
    tiny = 2.0 ** -9 * one[1].max()
    assert np.all(np.abs(d1 - x) <= np.maximum(2.0 ** -4 * np.abs(x), tiny / 2) * (1 + 1e-6))
    assert np.all(np.abs(d2 - x) <= 2 * np.maximum(2.0 ** -4 * np.abs(x), tiny / 2) * (1 + 2.0 ** -4))


def test_append_marks_what_is_not_finite_until_the_page_starts_again():
    x = np.ones((4, 1, 64), np.float32)
    pages, scale, table = np.zeros((1, 1, 32, 64), np.uint8), np.ones((1, 1)), np.array([[0]])
    x[1, 0, 3] = np.inf
    append(x, pages, scale, table, [0], [0, 4])
    assert np.isnan(scale[0, 0]) and not pages.any()
    append(np.ones((1, 1, 64)), pages, scale, table, [4], [0, 1])
    assert np.isnan(scale[0, 0])
    append(np.ones((1, 1, 64)), pages, scale, table, [0], [0, 1])
    assert scale[0, 0] == page_scale(1.0)


def test_limits():
    assert list(limits(3, 5, 0)) == [5, 5, 5]
    assert list(limits(3, 5, 1)) == [3, 4, 5]
    assert list(limits(5, 7, 2)) == [4, 4, 6, 6, 7]
    assert list(limits(4, 2, 1)) == [0, 0, 1, 2]         # more queries than keys: rows that see nothing
    o, a, s = attention(np.ones((4, 1, 64)), np.ones((2, 1, 64)), np.ones((2, 1, 64)), 1)
    assert not o[:2].any() and np.allclose(o[2:], 1.0)
    assert not attention(np.ones((2, 1, 64)), np.ones((0, 1, 64)), np.ones((0, 1, 64)))[0].any()


def test_codes_survive_decode_and_encode():
    c = np.array([i for i in range(256) if i & 0x7F != 0x7F], np.uint8)
    np.testing.assert_array_equal(e4m3_encode(e4m3_decode(c)), c)


# ---- refusals of the C entry points ----------------------------------------------------------
BUF = 4096   # an aligned address that a refused call never reads


def _rope(lib, dtype=0, x=BUF, xt=128, xh=64, out=BUF, ot=128, oh=64, tokens=1, heads=2, d=64, pos=BUF, pairs=(12, 10, 10),
          theta=1e4, half=0, inverse=0, naxes=None):
    arr = (ctypes.c_int32 * max(1, len(pairs)))(*pairs)
    return lib.la_op_rope_axes(dtype, x, xt, xh, out, ot, oh, tokens, heads, d, pos, len(pairs) if naxes is None else naxes, arr,
                               theta, half, inverse, None)


@pytest.mark.parametrize("over", [
    dict(dtype=3), dict(dtype=-1), dict(x=None), dict(out=None), dict(pos=None), dict(tokens=-1), dict(heads=0),
    dict(heads=65536, xt=1 << 30, ot=1 << 30), dict(d=0), dict(d=1), dict(d=257), dict(pairs=()), dict(pairs=(0, 0)),
    dict(pairs=(33,)), dict(pairs=(12, 10, 11)), dict(pairs=(-1, 3)), dict(pairs=(1, 1, 1, 1, 1)), dict(theta=0.5),
    dict(theta=float("nan")), dict(theta=float("inf")), dict(xh=63), dict(oh=0), dict(xt=-1), dict(ot=0, tokens=2),
    dict(ot=64, tokens=3), dict(ot=100, tokens=2, oh=64), dict(x=BUF + 1), dict(out=BUF + 1), dict(pos=BUF + 2), dict(dtype=1, x=BUF + 2), dict(naxes=-1),
])
def test_rope_axes_refuses(lib, over):
    assert _rope(lib, **over) == _lib.LA_EINVAL


def test_rope_axes_without_tokens_is_nothing(lib):
    assert _rope(lib, tokens=0, x=None, out=None, pos=None) == _lib.LA_OK


def _cache(**over):
    base = dict(k_pages=BUF, v_pages=BUF, k_scale=BUF, v_scale=BUF, block_table=BUF, num_pages=4, heads=2, page_tokens=64,
                head_dim=64, batch=2, max_pages=2)
    base.update({k: v for k, v in over.items() if k in base})
    return _lib.LaPagedCache(*base.values())


CACHE_BAD = [dict(k_pages=None), dict(v_pages=None), dict(k_scale=None), dict(v_scale=None), dict(block_table=None),
             dict(k_pages=BUF + 8), dict(v_pages=BUF + 4), dict(num_pages=0), dict(heads=0), dict(heads=65536),
             dict(page_tokens=16), dict(page_tokens=63), dict(page_tokens=256), dict(head_dim=96), dict(head_dim=256),
             dict(k_scale=BUF + 2), dict(v_scale=BUF + 1), dict(block_table=BUF + 2), dict(batch=0), dict(batch=65536),
             dict(max_pages=0), dict(max_pages=1 << 26)]


def _append(lib, cache=None, dtype=0, k=BUF, kt=128, kh=64, v=BUF, vt=128, vh=64, tokens=2, cu=BUF, lens=BUF, max_new=2,
            pos=BUF, pairs=(12, 10, 10), theta=1e4, half=0, **over):
    c = _cache(**over) if cache is None else cache
    arr = (ctypes.c_int32 * max(1, len(pairs)))(*pairs)
    return lib.la_op_cache_append_fp8(ctypes.byref(c), dtype, k, kt, kh, v, vt, vh, tokens, cu, lens, max_new, pos,
                                      len(pairs), arr, theta, half, None)


@pytest.mark.parametrize("over", CACHE_BAD + [
    dict(dtype=3), dict(k=None), dict(v=None), dict(cu=None), dict(lens=None), dict(pos=None), dict(tokens=-1),
    dict(max_new=-1), dict(kt=0), dict(kh=63), dict(vt=-1), dict(vh=1), dict(pairs=(33,)), dict(pairs=(0,)), dict(theta=0.0),
    dict(k=BUF + 1), dict(dtype=1, v=BUF + 2), dict(cu=BUF + 2), dict(lens=BUF + 1), dict(pos=BUF + 2),
])
def test_append_refuses(lib, over):
    assert _append(lib, **over) == _lib.LA_EINVAL


def test_append_of_nothing(lib):
    assert lib.la_op_cache_append_fp8(None, 0, BUF, 128, 64, BUF, 128, 64, 2, BUF, BUF, 2, None, 0, None, 1e4, 0,
                                      None) == _lib.LA_EINVAL
    assert _append(lib, tokens=0, k=None, v=None, pos=None) == _lib.LA_OK
    assert _append(lib, max_new=0) == _lib.LA_OK


def _attn(lib, dtype=0, q=BUF, qt=256, qh=64, tokens=2, q_heads=4, cu=BUF, lens=BUF, max_q=1, max_kv=128, causal=1, scale=0.1,
          out=BUF, ot=256, oh=64, out32=None, ws=BUF, ws_bytes=1 << 40, **over):
    c = _cache(**over)
    return lib.la_op_attention_cache_fp8(ctypes.byref(c), dtype, q, qt, qh, tokens, q_heads, cu, lens, max_q, max_kv, causal,
                                         scale, out, ot, oh, out32, ws, ws_bytes, None)


@pytest.mark.parametrize("over", CACHE_BAD + [
    dict(dtype=1), dict(dtype=3), dict(q=None), dict(out=None), dict(cu=None), dict(lens=None), dict(tokens=-1), dict(q_heads=3),
    dict(q_heads=0), dict(max_q=-1), dict(max_kv=-1), dict(causal=-1), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(qh=63), dict(qt=-1), dict(ot=0), dict(ot=64, oh=64), dict(ot=128, oh=64), dict(oh=66), dict(ot=258),
    dict(out=BUF + 4), dict(q=BUF + 1), dict(out32=BUF + 8), dict(max_kv=1 << 20, ws_bytes=0), dict(max_kv=1 << 20, ws=None),
    dict(max_kv=1 << 20, ws=BUF + 8), dict(cu=BUF + 2), dict(lens=BUF + 2),
])
def test_attention_refuses(lib, over):
    assert _attn(lib, **over) == _lib.LA_EINVAL


def test_attention_of_nothing_and_workspace(lib):
    assert _attn(lib, tokens=0, q=None, out=None) == _lib.LA_OK
    assert _attn(lib, max_q=0) == _lib.LA_OK
    c = _cache()
    w = lambda *a: lib.la_op_attention_cache_fp8_workspace(ctypes.byref(c), *a)  # noqa: E731
    assert w(2, 4, 1, 128) == 0                          # short keys are not split
    assert w(2, 4, 1, 1 << 20) > 0
    assert w(2, 3, 1, 128) == _lib.LA_EINVAL and w(-1, 4, 1, 128) == _lib.LA_EINVAL
    assert lib.la_op_attention_cache_fp8_workspace(None, 2, 4, 1, 128) == _lib.LA_EINVAL


def test_binding_refuses_what_is_not_on_a_gpu():
    import torch
    from streaming_causal_video_timestep_b200 import op_attention_cache_fp8, op_cache_append_fp8, op_rope_axes
    x, pos = torch.zeros(2, 2, 64), torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(TypeError):
        op_rope_axes(x, pos, (12, 10, 10))
    with pytest.raises(TypeError):
        op_cache_append_fp8(x, x, None, None, None, None, None, None, None, 1)
    with pytest.raises(TypeError):
        op_attention_cache_fp8(x, None, None, None, None, None, None, None, 1, 1)


def test_waits_of_the_attention_kernel_are_decided_by_the_warp():
    """A bounded wait may end differently from lane to lane (each looks at the clock, and at the CTA's abort flag, by
    itself), and what follows it needs the whole warp: every answer, and every look at the flag, goes through a vote."""
    import os
    import re
    src = os.path.join(os.path.dirname(_lib.__file__), "csrc", "attn_cache_tc.cu")
    text = re.sub(r"//[^\n]*", "", open(src).read())
    seen = 0
    for s in re.split(r"[;{}]", text):
        s = " ".join(s.split())
        reads = re.search(r"\babort_flag\b(?! = )", s) and "volatile" not in s
        if "mbar_wait(" not in s and not reads:
            continue
        seen += 1
        alone = re.match(r"(for \([^)]*\) )?(if \(!ok && t > 1\) )?mbar_wait\(", s)    # nothing depends on its answer
        assert alone or re.search(r"__all_sync\(0xffffffffu, [^;]*(mbar_wait|abort_flag)", s), s
        if not alone:
            vote = s.index("__all_sync(")
            assert all(m.start() > vote for m in re.finditer(r"mbar_wait\(|\babort_flag\b", s)), s
            depth, end = 0, vote + len("__all_sync")
            while True:                                            # the vote's own parentheses hold all of them
                depth += {"(": 1, ")": -1}.get(s[end], 0)
                end += 1
                if depth == 0:
                    break
            assert not re.search(r"mbar_wait\(|\babort_flag\b", s[end:]), s
    assert seen >= 7


def test_local_arrays_read_as_vectors_are_aligned():
    """A local array that is read or written as 8- or 16-byte vectors has to be declared with that alignment: its
    element type alone does not give it."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(_lib.__file__), "csrc")
    bad = []
    for name in sorted(os.listdir(csrc)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(csrc, name)).read())
        for m in re.finditer(r"^[ \t]*((?:T|TO|__half|__nv_bfloat16|u?int(?:8|16|32)_t|float|unsigned(?: char| short)?) (\w+)(?:\[\w+\])+);", text, re.M):
            use = re.search(r"reinterpret_cast<(?:const )?(?:uint2|uint4|float4|longlong2)\*>\(&?" + m[2] + r"\b", text[m.end():].split("\n}", 1)[0])   # to the function's end
            if use:
                bad.append(f"{name}: {m[1]}")
    assert not bad, bad


def test_outputs_whose_rows_overlap_are_refused_at_any_stride(lib):
    """Strides whose products pass 64 bits: rows 2^40 apart, as are the heads, lie over one another."""
    far = 1 << 40
    assert _rope(lib, tokens=1 << 30, heads=3, xt=far, xh=far, ot=far, oh=far) == _lib.LA_EINVAL
    assert _attn(lib, tokens=1 << 30, q_heads=(1 << 26) + 2, qt=far, qh=far, ot=far, oh=far, ws_bytes=1 << 62) == _lib.LA_EINVAL
