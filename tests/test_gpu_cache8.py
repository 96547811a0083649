"""Rotary positions with several axes, the paged 8-bit cache and attention over it on the GPU, against the oracle's
definitions in 64 bits (oracle/cache8.py) on the same inputs.

Tolerances (u = 2^-24, eps_t the type's epsilon):
  rotation   an angle is a fraction of a turn exact to 2^-32 (1.5e-9 rad); its rest within an eighth of a turn goes to
             fp32 and is scaled there (3 u of at most pi/4: 1.4e-7 rad), the series and its evaluation add 2 u and 3e-9;
             the two products and the sum add 3 u: together at most TURN * (|x0| + |x1|) with TURN = 5.2e-7, plus half a
             step of the output.
  append     V's scales and codes are integer decisions on the input: equal.  A rotated K lies within the rotation's
             bound of the exact one: its value is off by half an e4m3 step plus that, and its scale is the exact one's
             unless the page's largest magnitude is within the bound of 448 * 2^e.
  attention  q (under a power of two) and the codes are exact in fp16.  With S the largest sum of |q||k| terms of a
             row's scores, a score is off by (d + 4) u S, exp2 and its argument add 4 u of the result and of |score|
             <= S: each P by a factor 1 +- 2 ((d + 8) u S + 4 u), and fp16 rounds it by 2^-11; a sum of L terms in fp32
             whose additions come in steps of 16 keys is off by (L / 16 + 64) 2 u.  All relative to a = sum p |v|, in
             numerator and normaliser; P below 2^-25 of the largest (times the value scales) may vanish: L 2^-30 max|v|.
"""
import numpy as np
import pytest

from oracle.cache8 import append, attention, dense_cache, page_scale, rotate_axes
from oracle.fp8 import e4m3_decode

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
TURN = 5.2e-7
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
PAIRS = {128: (22, 21, 21), 64: (12, 10, 10)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from streaming_causal_video_timestep_b200 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    yield
    assert status() == 0


def status():
    from streaming_causal_video_timestep_b200 import load
    return load().la_op_status(None)


def rand(seed, *shape, dtype="bf16"):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32)).cuda().to(DT[dtype])


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def np64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def half_step(ref, dt):
    f = torch.finfo(dt)
    return np.maximum(np.abs(ref) * (f.eps / 2), f.smallest_normal * f.eps / 2)


def turn_bound(x, pairs, half):
    """TURN * (|x0| + |x1|) at every rotated element, 0 at the others."""
    n, a = sum(pairs), np.abs(x)
    lo, hi = (slice(0, n), slice(n, 2 * n)) if half else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    b = np.zeros_like(a)
    b[..., lo] = b[..., hi] = TURN * (a[..., lo] + a[..., hi])
    return b


def near(got, ref, bound, what=""):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.abs(got - ref)[bad].max():.3e} against {np.broadcast_to(bound, bad.shape)[bad].max():.3e}"


# ---- rotary positions ------------------------------------------------------------------------
ROPE = [(7, 3, 128, (22, 21, 21)), (1, 1, 64, (12, 10, 10)), (300, 40, 128, (22, 21, 21)), (33, 5, 64, (32,)),
        (65, 2, 128, (16, 8)), (9, 2, 40, (7, 6, 4)), (5, 3, 7, (1, 2)), (4, 2, 256, (32, 32, 32, 32)), (11, 1, 2, (1,))]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("T,H,d,pairs", ROPE)
def test_rope_axes(T, H, d, pairs, half, dtype):
    from streaming_causal_video_timestep_b200 import op_rope_axes
    x = rand(T + d, T, H, d, dtype=dtype)
    pos = np.random.default_rng(3).integers(-2000, 90000, (T, len(pairs)))
    for inverse in (False, True):
        y = op_rope_axes(x, i32(pos), pairs, half=half, inverse=inverse)
        ref = rotate_axes(np64(x), pos, pairs, half=half, inverse=inverse)
        # the oracle's fp64 angle pos * omega is itself rounded: 2^-53 * 9e4 rad, far below TURN
        near(np64(y), ref, turn_bound(np64(x), pairs, half) + half_step(ref, x.dtype) * (1 + 1e-5), f"inverse={inverse}")
        n = 2 * sum(pairs)
        assert torch.equal(y[..., n:], x[..., n:])


def test_rope_axes_at_every_int32_position():
    from streaming_causal_video_timestep_b200 import op_rope_axes
    pos = np.array([[2 ** 31 - 1, 0, 0], [-2 ** 31, 1, -1], [1 << 24, (1 << 24) + 1, -(1 << 30)], [0, 0, 0]])
    x = rand(0, 4, 2, 128, dtype="fp32")
    y = np64(op_rope_axes(x, i32(pos), PAIRS[128]))
    # angles by integer arithmetic: a power of theta with 40 digits, reduced modulo a turn exactly
    from fractions import Fraction
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    pi2 = Decimal("6.28318530717958647692528676655900576839433879875021164194989")
    n, ang = sum(PAIRS[128]), np.zeros((4, 64))
    col = 0
    for a, p in enumerate(PAIRS[128]):
        for j in range(p):
            turns = Fraction(Decimal(10000) ** (Decimal(-j) / Decimal(p)) / pi2)
            for t in range(4):
                f = (int(pos[t, a]) * turns) % 1
                ang[t, col] = float(f) * 2 * np.pi
            col += 1
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    v = np64(x)
    ref = np.empty_like(v)
    ref[..., 0::2] = v[..., 0::2] * c - v[..., 1::2] * s
    ref[..., 1::2] = v[..., 0::2] * s + v[..., 1::2] * c
    # the table's 2^-65 turns a position step: 2^31 * 2^-65 turns = 3.7e-10 rad on top
    near(y, ref, turn_bound(v, PAIRS[128], False) * (1 + 1e-2) + half_step(ref, torch.float32) * 1.01)
    assert np.array_equal(y[3], v[3])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("half", [False, True])
def test_rope_axes_strides_and_in_place(half, dtype):
    from streaming_causal_video_timestep_b200 import op_rope_axes
    T, H, d = 37, 4, 128
    pos = np.random.default_rng(3).integers(0, 900, (T, 3))
    qkv = rand(5, T, 3 * H, d, dtype=dtype)
    ref = op_rope_axes(qkv[:, :2 * H].contiguous(), i32(pos), PAIRS[d], half=half)
    planes = qkv[:, :2 * H].transpose(0, 1).contiguous().transpose(0, 1)          # [H, T, d] storage
    assert torch.equal(op_rope_axes(planes, i32(pos), PAIRS[d], half=half), ref)
    odd = torch.zeros(T, 2 * H, d + 3, dtype=DT[dtype], device="cuda")            # rows that are not 16-byte aligned
    odd[..., 1:d + 1] = qkv[:, :2 * H]
    assert torch.equal(op_rope_axes(odd[..., 1:d + 1], i32(pos), PAIRS[d], half=half), ref)
    out = torch.full((T, 2 * H, d + 3), 7.0, dtype=DT[dtype], device="cuda")
    op_rope_axes(qkv[:, :2 * H], i32(pos), PAIRS[d], half=half, out=out[..., 2:d + 2])
    assert torch.equal(out[..., 2:d + 2], ref) and (out[..., :2] == 7).all() and (out[..., d + 2:] == 7).all()
    v = qkv[:, 2 * H:].clone()
    view = qkv[:, :2 * H]
    assert op_rope_axes(view, i32(pos), PAIRS[d], half=half, out=view) is view     # in place, q and k at once
    assert torch.equal(view, ref) and torch.equal(qkv[:, 2 * H:], v)
    back = op_rope_axes(ref, i32(pos), PAIRS[d], half=half, inverse=True)
    x = rand(5, T, 3 * H, d, dtype=dtype)[:, :2 * H]
    # there and back: the bound of each rotation, and the first one's rounding turned back
    r0, r1 = np64(x), np64(ref)
    step = turn_bound(r0, PAIRS[d], half) + turn_bound(r1, PAIRS[d], half) + half_step(r0, DT[dtype])
    step = step + (turn_bound(half_step(r1, DT[dtype]), PAIRS[d], half) / TURN)
    near(np64(back), r0, step * 1.01)


def test_rope_axes_of_no_tokens_and_refusals():
    from streaming_causal_video_timestep_b200 import LaError, op_rope_axes
    x, pos = rand(0, 4, 2, 64), i32(np.zeros((4, 3)))
    assert op_rope_axes(x[:0], pos[:0], PAIRS[64]).shape == (0, 2, 64)
    for bad in (dict(pos=pos.long()), dict(pos=pos[:3]), dict(pos=pos[:, :2]), dict(x=x.transpose(1, 2)), dict(x=x.double()),
                dict(out=x[:3]), dict(out=x.float()), dict(pos=pos.t().contiguous().t())):
        with pytest.raises(ValueError):
            op_rope_axes(**{"x": x, "pos": pos, "pairs": PAIRS[64], **bad})
    for bad in (dict(x=x[0]), dict(pos=pos.cpu()), dict(x=x.cpu())):
        with pytest.raises(TypeError):
            op_rope_axes(**{"x": x, "pos": pos, "pairs": PAIRS[64], **bad})
    for bad in (dict(pairs=(12, 10, 11)), dict(theta=0.0), dict(x=x[:, :1].expand(4, 2, 64))):
        with pytest.raises(LaError):
            op_rope_axes(**{"x": x, "pos": pos, "pairs": PAIRS[64], **bad})


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("half,inverse", [(False, False), (True, False), (False, True)])
def test_rope_axes_gradient(half, inverse, dtype):
    """The gradient is the rotation turned back: within the rotation's bound and one rounding of the definition; a
    gradient that arrives expanded, transposed or strided gives the same."""
    from streaming_causal_video_timestep_b200 import op_rope_axes
    T, H, d, pairs = 13, 3, 128, (20, 21, 6)
    pos = np.random.default_rng(5).integers(-300, 9000, (T, 3))
    x = rand(11, T, H, d, dtype=dtype).requires_grad_()
    y = op_rope_axes(x, i32(pos), pairs, half=half, inverse=inverse)
    assert y.requires_grad and torch.equal(y.detach(), op_rope_axes(x.detach(), i32(pos), pairs, half=half, inverse=inverse))
    wide = rand(12, T, H, d + 4, dtype=dtype)
    for g in (rand(13, T, H, d, dtype=dtype), wide[..., 1:d + 1], rand(14, H, T, d, dtype=dtype).transpose(0, 1),
              rand(15, T, d, H, dtype=dtype).transpose(1, 2), rand(16, 1, 1, d, dtype=dtype).expand(T, H, d),
              torch.ones((), dtype=DT[dtype], device="cuda").expand(T, H, d)):
        (dx,) = torch.autograd.grad(y, x, g, retain_graph=True)
        ref = rotate_axes(np64(g), pos, pairs, half=half, inverse=not inverse)
        near(np64(dx), ref, turn_bound(np64(g), pairs, half) + half_step(ref, x.dtype) * (1 + 1e-5))
        assert dx.dtype == x.dtype
    y.backward(g)
    y2 = op_rope_axes(x, i32(pos), pairs, half=half, inverse=inverse)
    y2.backward(g)                                       # accumulates: twice the same
    assert torch.equal(x.grad, (dx.float() * 2).to(x.dtype))


def test_rope_axes_gradient_against_differences():
    from streaming_causal_video_timestep_b200 import op_rope_axes
    T, H, d = 4, 2, 64
    pos, pairs = i32(np.random.default_rng(6).integers(0, 4000, (T, 2))), (9, 14)
    x, w = rand(17, T, H, d, dtype="fp32").requires_grad_(), rand(18, T, H, d, dtype="fp32")
    f = lambda v: float((op_rope_axes(v, pos, pairs).double() * w.double()).sum())  # noqa: E731
    (dx,) = torch.autograd.grad(op_rope_axes(x, pos, pairs), x, w)
    for i in ((0, 0, 0), (1, 1, 1), (2, 0, 17), (3, 1, 45), (3, 0, 46), (1, 0, 63)):
        e = torch.zeros_like(x)
        e[i] = 1.0
        with torch.no_grad():
            got = (f(x + e) - f(x - e)) / 2              # linear in x: only the two outputs that it moves are rounded
        # x +- e rounds once (|x| < 8: 4 u), the output's bound is TURN (|x0| + |x1|) + u |y| at both of the pair, at both ends
        bound = 2 * (2 * 16 * TURN + 16 * U + 8 * U) * float(w.abs().max())
        assert abs(got - float(dx[i])) <= bound + TURN * 16
    # twice: the gradient of the gradient is the rotation itself
    g = rand(19, T, H, d, dtype="fp32").requires_grad_()
    (dx,) = torch.autograd.grad(op_rope_axes(x, pos, pairs), x, g, create_graph=True)
    (dg,) = torch.autograd.grad(dx, g, w)
    assert torch.equal(dg, op_rope_axes(w, pos, pairs))


def test_rope_axes_gradient_streams_graphs_and_refusals():
    from streaming_causal_video_timestep_b200 import op_rope_axes
    pos = i32(np.arange(300).reshape(100, 3))
    x, g = rand(20, 100, 4, 128).requires_grad_(), rand(21, 100, 4, 128)
    (want,) = torch.autograd.grad(op_rope_axes(x, pos, PAIRS[128]), x, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = op_rope_axes(x, pos, PAIRS[128], stream=side)    # runs on side, and so does its backward
    torch.cuda.current_stream().wait_stream(side)
    (got,) = torch.autograd.grad(y, x, g)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (out,) = torch.autograd.grad(op_rope_axes(x, pos, PAIRS[128]), x, g)
    g.copy_(rand(22, 100, 4, 128))
    graph.replay()
    (want,) = torch.autograd.grad(op_rope_axes(x, pos, PAIRS[128]), x, g)
    assert torch.equal(out, want)
    from types import SimpleNamespace
    for v in (x, x.detach()):
        with pytest.raises(ValueError, match="stream is on"):
            op_rope_axes(v, pos, PAIRS[128], stream=SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0))
    for out in (torch.empty_like(x), x):
        with pytest.raises(ValueError, match="gradient"):
            op_rope_axes(x, pos, PAIRS[128], out=out)
    with torch.no_grad():
        y = op_rope_axes(x, pos, PAIRS[128], out=torch.empty_like(x))
    assert not y.requires_grad and not op_rope_axes(x.detach(), pos, PAIRS[128]).requires_grad
    y = op_rope_axes(x, pos, PAIRS[128])
    pos += 1                                             # positions that changed since: refused, not a wrong gradient
    with pytest.raises(RuntimeError):
        torch.autograd.grad(y, x, g)


# ---- the cache ---------------------------------------------------------------------------------
class Cache:
    """A paged cache on the GPU and the oracle's copy of it."""

    def __init__(self, seed, batch, width, heads, page, d, spare=2):
        rng = np.random.default_rng(seed)
        num = batch * width + spare
        self.table = rng.permutation(num)[:batch * width].reshape(batch, width)
        self.page, self.heads, self.d = page, heads, d
        # stale codes everywhere, NaN codes among them, and stale scales: what an append does not write is not seen
        self.k, self.v = (rng.integers(0, 256, (num, heads, page, d)).astype(np.uint8) for _ in range(2))
        self.ks, self.vs = (2.0 ** rng.integers(-9, 3, (num, heads)) for _ in range(2))
        self.ks[self.table.reshape(-1)[-1]] = np.nan
        self.g = [torch.from_numpy(a).cuda() for a in (self.k, self.v)] + [
            torch.from_numpy(a.astype(np.float32)).cuda() for a in (self.ks, self.vs)] + [i32(self.table)]

    def append(self, k, v, lens, cu, max_new=None, pos=None, pairs=None, half=False, **kw):
        from streaming_causal_video_timestep_b200 import op_cache_append_fp8
        p = None if pos is None else i32(pos)
        op_cache_append_fp8(k, v, *self.g, i32(lens), i32(cu), int(max(np.diff(cu))) if max_new is None else max_new, pos=p,
                            pairs=pairs, half=half, **kw)
        kk = np64(k) if pos is None else rotate_axes(np64(k), pos, pairs, half=half)
        append(kk, self.k, self.ks, self.table, lens, cu)
        append(np64(v), self.v, self.vs, self.table, lens, cu)

    def check_v(self):
        np.testing.assert_array_equal(self.g[3].cpu().numpy().astype(np.float64), self.vs)
        np.testing.assert_array_equal(self.g[1].cpu().numpy(), self.v)


def lens_of(kind, batch, top):
    if kind == "one":
        return [1] * batch
    if kind == "even":
        return [top] * batch
    return [0 if i == 1 else max(1, top - 13 * i) for i in range(batch)]       # ragged, one of them empty


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("page,d", [(32, 64), (64, 128), (128, 128), (128, 64)])
@pytest.mark.parametrize("kind,top", [("one", 1), ("ragged", 150), ("even", 64)])
def test_append(kind, top, page, d, dtype):
    B, H = 3, 3
    new, old = lens_of(kind, B, top), [0, page - 1, 2 * page + 5]
    cu = np.concatenate([[0], np.cumsum(new)])
    c = Cache(7, B, (top + 2 * page + 5) // page + 1, H, page, d)
    N = cu[-1] + 3                                                             # rows behind the last sequence
    k, v = rand(1, N, H, d, dtype=dtype), rand(2, N, H, d, dtype=dtype)
    k[cu[-1]:] = v[cu[-1]:] = float("nan")
    c.append(k, v, old, cu)                                                    # not rotated: K is exact, too
    c.check_v()
    np.testing.assert_array_equal(c.g[0].cpu().numpy(), c.k)
    np.testing.assert_array_equal(c.g[2].cpu().numpy().astype(np.float64), c.ks)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("page,d,pairs,dtype", [(32, 64, (12, 10, 10), "bf16"), (64, 128, (22, 21, 21), "fp16"),
                                                (128, 128, (8, 16), "fp32"), (64, 64, (9, 4), "bf16"),
                                                (64, 128, (5, 6, 7), "fp32")])
def test_append_rotates(page, d, pairs, dtype, half):
    B, H, new, old = 2, 3, [page + 9, 41], [3, page]
    cu = np.concatenate([[0], np.cumsum(new)])
    c = Cache(8, B, 4, H, page, d)
    c.ks[:] = c.vs[:] = 2.0 ** -20                                             # the new tokens set every scale
    c.g[2].fill_(2.0 ** -20), c.g[3].fill_(2.0 ** -20)
    k, v = rand(1, cu[-1], H, d, dtype=dtype), rand(2, cu[-1], H, d, dtype=dtype)
    pos = np.random.default_rng(4).integers(-50, 40000, (cu[-1], len(pairs)))
    c.append(k, v, old, cu, pos=pos, pairs=pairs, half=half)
    c.check_v()
    exact, bound = rotate_axes(np64(k), pos, pairs, half=half), turn_bound(np64(k), pairs, half)
    scale, codes = c.g[2].cpu().numpy().astype(np.float64), c.g[0].cpu().numpy()
    for b in range(B):
        for t in range(new[b]):
            j, row = old[b] + t, cu[b] + t
            pg = c.table[b, j // page]
            for h in range(H):
                if scale[pg, h] != c.ks[pg, h]:                                # only at the border, by one step
                    rows = [cu[b] + i for i in range(new[b]) if (old[b] + i) // page == j // page]
                    lo = page_scale((np.abs(exact[rows, h]) - bound[rows, h]).max())
                    hi = page_scale((np.abs(exact[rows, h]) + bound[rows, h]).max())
                    assert scale[pg, h] in (lo, hi)
            s = scale[pg][:, None]
            got = e4m3_decode(codes[pg, :, j % page]) * s
            near(got, exact[row], np.maximum(2.0 ** -4 * (np.abs(exact[row]) + bound[row]), 2.0 ** -10 * s) + bound[row])


def test_append_grows_scales_and_restarts_pages():
    page, d, H = 64, 128, 2
    c = Cache(9, 1, 3, H, page, d)
    at = 0
    for step, n in enumerate((1, 1, 30, 1, 40, 1, 17)):                        # magnitudes grow and shrink from call to call
        k, v = rand(step, n, H, d) * 2.0 ** (3 * (step % 3) - 4), rand(step + 50, n, H, d) * 2.0 ** (2 * step)
        c.append(k, v, [at], [0, n])
        c.check_v()
        np.testing.assert_array_equal(c.g[0].cpu().numpy(), c.k)
        at += n
    c.append(rand(77, 3, H, d) * 1e-3, rand(78, 3, H, d), [0], [0, 3])         # the first page is written again
    c.check_v()
    np.testing.assert_array_equal(c.g[0].cpu().numpy(), c.k)


def test_append_of_extremes():
    page, d, H = 32, 64, 3
    c = Cache(10, 2, 2, H, page, d)
    v = torch.zeros(8, H, d, device="cuda")
    v[0, 1, :4] = torch.tensor([3.4e38, -3.4e38, 1e-38, 448.0])
    v[1, 2, :4] = torch.tensor([448.0, 447.9999, 1e-45, -2.0 ** -64])
    v[5, 0, 1] = float("inf")
    v[6, 1, 2] = float("nan")
    c.append(v, v, [0, 0], [0, 4, 8])
    c.check_v()
    np.testing.assert_array_equal(c.g[0].cpu().numpy(), c.k)
    c.append(v[:1], v[:1], [4, 4], [0, 0, 1])                                  # a page that was marked stays marked
    c.check_v()
    assert np.isnan(c.g[3][c.table[1, 0]].cpu().numpy()).tolist() == [True, True, False]


def test_append_strides():
    page, d, H = 64, 128, 3
    a, b = Cache(11, 1, 3, H, page, d), Cache(11, 1, 3, H, page, d)
    qkv = rand(3, 100, 3 * H, d)
    odd = torch.zeros(100, H, d + 1, dtype=torch.bfloat16, device="cuda")
    odd[..., 1:] = qkv[:, 2 * H:]
    pos = np.arange(300).reshape(100, 3)
    for half in (False, True):
        a.append(qkv[:, H:2 * H], qkv[:, 2 * H:], [7], [0, 100], pos=pos, pairs=PAIRS[d], half=half)
        b.append(qkv[:, H:2 * H].transpose(0, 1).contiguous().transpose(0, 1), odd[..., 1:], [7], [0, 100], pos=pos,
                 pairs=PAIRS[d], half=half)
        a.check_v()
        for x, y in zip(a.g, b.g):
            assert torch.equal(x.nan_to_num(5) if x.is_floating_point() else x, y.nan_to_num(5) if y.is_floating_point() else y)


def test_append_leaves_out_what_does_not_fit():
    from streaming_causal_video_timestep_b200 import _lib
    page, d, H, B = 32, 64, 2, 3
    k = rand(1, 12, H, d)
    for lens, cu, table, max_new in (([0, 50, 0], [0, 4, 20, 12], None, 20),        # past the rows, and falling
                                     ([0, -1, 0], [0, 4, 8, 12], None, 4),
                                     ([0, 61, 0], [0, 4, 8, 12], None, 4),          # past the table's pages
                                     ([0, 5, 0], [0, 4, 9, 12], None, 4),           # more than max_new
                                     ([0, 5, 0], [0, 4, 8, 12], (1, 0, 999), 4),    # a page that is not there
                                     ([0, 5, 0], [0, 4, 8, 12], (1, 0, -1), 4)):
        c = Cache(12, B, 2, H, page, d)
        keep = c.g[1].clone()
        if table:
            c.g[4][table[0], table[1]] = table[2]
        from streaming_causal_video_timestep_b200 import op_cache_append_fp8
        op_cache_append_fp8(k, k, *c.g, i32(lens), i32(cu), max_new)
        assert status() == _lib.LA_EDEVICE and status() == _lib.LA_OK
        assert torch.equal(c.g[1][c.table[1].tolist()], keep[c.table[1].tolist()])
        assert not torch.equal(c.g[1][c.table[0, 0]], keep[c.table[0, 0]])          # the first sequence is appended


# ---- attention -----------------------------------------------------------------------------------
def attend(c, q, kv, cu, causal=0, max_q=None, max_kv=None, scale=None, out=None, stream=None):
    from streaming_causal_video_timestep_b200 import op_attention_cache_fp8
    o32 = torch.full(q.shape, 9.0, dtype=torch.float32, device="cuda")
    out = op_attention_cache_fp8(q, *c.g, i32(kv), i32(cu), int(max(np.diff(cu))) if max_q is None else max_q,
                                 max(kv) if max_kv is None else max_kv, causal_block=causal, scale=scale, out=out, out32=o32,
                                 stream=stream)
    return out, o32


def check_attention(c, q, kv, cu, causal=0, scale=None, **kw):
    out, o32 = attend(c, q, kv, cu, causal, scale=scale, **kw)
    pages, scales = [t.cpu().numpy() for t in c.g[:2]], [t.cpu().numpy() for t in c.g[2:4]]
    d = q.shape[2]
    for b in range(len(kv)):
        rows = slice(cu[b], cu[b + 1])
        k, v = (dense_cache(pages[i], scales[i], c.table, b, kv[b]) for i in range(2))
        ref, a, s = attention(np64(q[rows]), k, v, causal, scale)
        L = kv[b]
        p_err = 2 * ((d + 8) * U * s + 4 * U)
        bound = a * (2.0 ** -11 + 2 * p_err + 2 * (L / 16 + 64) * 2 * U) + L * 2.0 ** -30 * np.abs(v).max(initial=0.0)
        near(np64(o32[rows]), ref, bound, f"out32 of sequence {b}")
        near(np64(out[rows]), ref, bound * 1.01 + half_step(ref, q.dtype) * 1.01, f"out of sequence {b}")
    assert (o32[cu[-1]:] == 9).all()
    return out


def filled(seed, B, lens, H, page, d, spread=1.0):
    """A cache whose first lens[b] tokens were appended (values of several magnitudes from page to page)."""
    c = Cache(seed, B, max(1, -(-max(lens) // page)) + 1, H, page, d)
    n = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    grow = torch.exp2(torch.from_numpy(np.random.default_rng(seed).integers(-3, 3, (max(n, 1), 1, 1)) // 2 * 2.0).cuda())[:n]
    if n:
        c.append((rand(seed + 1, n, H, d, dtype="fp32") * spread), (rand(seed + 2, n, H, d, dtype="fp32") * grow).float(), [0] * B, cu)
    return c


SHAPES = [  # batch lens of keys, queries, key heads, group, page, d, causal
    ([1], [1], 1, 1, 64, 128, 1), ([1], [1], 2, 3, 32, 64, 0), ([17, 0, 130], [1, 1, 1], 2, 4, 64, 128, 1),
    ([1000, 333], [1, 1], 3, 1, 64, 128, 0), ([4097], [1], 1, 8, 128, 64, 1), ([700, 65, 64], [3, 5, 1], 2, 5, 64, 128, 1),
    ([129, 40], [16, 7], 1, 1, 32, 128, 1), ([300], [130], 2, 2, 64, 128, 1), ([257, 0, 31], [200, 5, 31], 2, 1, 32, 64, 7),
    ([390], [257], 1, 3, 128, 128, 0), ([50, 128], [64, 300], 1, 2, 64, 64, 1), ([512], [256], 2, 1, 64, 128, 128),
    ([1300], [513], 1, 2, 128, 64, 100), ([64, 640], [0, 384], 2, 1, 64, 128, 192), ([33, 70], [17, 16], 2, 1, 32, 64, 1),
    ([200], [5], 1, 3, 64, 64, 2), ([96, 97, 95], [2, 1, 2], 1, 8, 32, 128, 1), ([128], [128], 1, 2, 128, 128, 1),
    ([140], [129], 1, 2, 64, 128, 1000), ([2, 1], [300, 20], 1, 1, 64, 128, 3),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kv,nq,Hk,G,page,d,causal", SHAPES)
def test_attention(kv, nq, Hk, G, page, d, causal, dtype):
    c = filled(20, len(kv), kv, Hk, page, d)
    cu = np.concatenate([[0], np.cumsum(nq)])
    q = rand(30, cu[-1] + 2, Hk * G, d, dtype=dtype)
    check_attention(c, q, kv, cu, causal)


@pytest.mark.parametrize("nq", [1, 9, 150])
def test_attention_split_long_keys(nq):
    """The key axis is split: pieces of several CTAs are joined, and the result does not depend on the bound max_kv."""
    c = filled(21, 1, [9000], 1, 64, 128)
    q = rand(31, nq, 2, 128)
    a = check_attention(c, q, [9000], [0, nq], 1)
    b, _ = attend(c, q, [9000], [0, nq], 1, max_kv=0)                          # not split
    near(np64(a), np64(b), np.abs(np64(b)) * 2.0 ** -7 + 2.0 ** -12 * 8)       # two bf16 roundings of values 2^-11 (a <= 8) apart
    for _ in range(3):
        assert torch.equal(attend(c, q, [9000], [0, nq], 1)[0], a)             # the same bits every time


@pytest.mark.parametrize("nq,max_kv", [(1, 3000), (1, 10 ** 6), (8, 700), (150, 2000), (150, 10 ** 6)])
def test_attention_whatever_the_bound_says(nq, max_kv):
    """max_kv below the length (the last piece takes the rest) and far above it (most pieces are empty)."""
    c = filled(26, 2, [5000, 90], 1, 32, 64)
    check_attention(c, rand(32, 2 * nq, 2, 64), [5000, 90], [0, nq, 2 * nq], 1, max_kv=max_kv)


def test_attention_rows_of_no_sequence():
    """A buffer much longer than the batch: its other rows are left alone and cost no workspace."""
    from streaming_causal_video_timestep_b200 import load
    c = filled(27, 1, [3000], 1, 64, 64)
    q = rand(33, 5000, 1, 64)
    out = torch.full_like(q, 3.0)
    check_attention(c, q, [3000], [0, 1], 1, out=out)
    assert (out[1:] == 3).all() and load() is not None


@pytest.mark.parametrize("kv,nq,Hk,G,d,causal", [
    ([1100], [300], 80, 1, 64, 1), ([2100], [130], 80, 4, 64, 0), ([1100], [300], 80, 1, 128, 100),
    ([1200, 700, 1100], [300, 300, 40], 30, 1, 128, 1), ([1100, 1100, 1100], [300, 0, 300], 30, 1, 64, 1),
    ([1030, 0, 1500], [290, 17, 5], 40, 1, 64, 0)])
def test_attention_of_more_units_than_sms(kv, nq, Hk, G, d, causal):
    """More than 148 units of 256 rows: the first round is whole, the rest in pieces, some of their units empty.  Rows of
    no sequence are left alone, and pieces or not, an element is within both bounds."""
    pairs = -(-max(nq) * G // 256)
    units = pairs * Hk * len(kv)
    assert units > 148 and units % 148 and max(kv) > 8 * 128
    c = filled(29, len(kv), kv, Hk, 64, d)
    cu = np.concatenate([[0], np.cumsum(nq)])
    q = rand(34, cu[-1] + 3, Hk * G, d)
    out = torch.full_like(q, 3.0)
    check_attention(c, q, kv, cu, causal, out=out)
    assert (out[cu[-1]:] == 3).all()
    again, _ = attend(c, q, kv, cu, causal)
    assert torch.equal(again[:cu[-1]], out[:cu[-1]])


def test_workspace_does_not_grow_with_rows_of_no_sequence():
    import ctypes
    from streaming_causal_video_timestep_b200 import _lib, load
    c = _lib.LaPagedCache(4096, 4096, 4096, 4096, 4096, 64, 2, 64, 64, 3, 64)
    need = lambda tokens, heads, max_q, max_kv: load().la_op_attention_cache_fp8_workspace(  # noqa: E731
        ctypes.byref(c), tokens, heads, max_q, max_kv)
    assert need(1, 2, 1, 3000) == need(5000, 2, 1, 3000) > 0
    assert need(300, 2, 300, 3000) == need(5000, 2, 300, 3000) > 0
    assert need(3, 2, 5000, 3000) == need(3, 2, 3, 3000) > 0               # no sequence has more rows than there are
    q = rand(35, 3, 2, 64)                                                  # and the call agrees: max_q above the rows
    f = filled(36, 1, [3000], 2, 64, 64)
    check_attention(f, q, [3000], [0, 3], 1, max_q=5000)


@pytest.mark.parametrize("nq,G", [(1, 1), (1, 4), (40, 2)])
def test_attention_peaked_and_far_apart(nq, G):
    """One key far above the rest, late (the running maximum moves) and early, and rows of q of very different sizes."""
    d, L = 128, 700
    c = Cache(22, 1, L // 64 + 1, 1, 64, d)
    k, v = rand(1, L, 1, d, dtype="fp32"), rand(2, L, 1, d, dtype="fp32")
    k[650] *= 30
    k[3] *= 20
    v[100:200] *= 2.0 ** 12
    c.append(k, v, [0], [0, L])
    q = rand(3, nq, G, d, dtype="fp32")
    q[0] *= 2.0 ** -20
    if nq > 2:
        q[1] *= 20
        q[2] *= 0
    check_attention(c, q.bfloat16(), [L], [0, nq], 0)
    check_attention(c, q.bfloat16(), [L], [0, nq], 0, scale=1e-3)


@pytest.mark.parametrize("tilt", [False, True])
@pytest.mark.parametrize("max_kv", [0, 5000])
@pytest.mark.parametrize("page,d", [(64, 128), (32, 64), (128, 128), (32, 128)])
@pytest.mark.parametrize("nq,G", [(1, 1), (3, 4), (150, 2)])
def test_attention_value_scales_far_apart(nq, G, page, d, max_kv, tilt):
    """Pages of zeros (scale 2^-64) beside values up to 1e37 (2^116), in every order, whole and in pieces; tilt: the
    large values lie where the weights are smallest.  Every key counts in the normaliser.

    The bound is the module's, with two changes.  An argument of an exponential is a score and log2 of a scale, of
    magnitude S + 128 at most, rounded three times (with the scale, the maximum, and where the scale is taken out
    again): 3 * 128 u ln 2 < 300 u more a P.  And P, stored with 2^-24 for its last place under a maximum M of
    score + log2 scale, is off by 2^-25 2^(M - 7) at most; M is no larger than the largest p_j vs_j, so
    L * 2^-32 * 448 * max_j p_j vs_j."""
    L = 11 * page - 7
    grade = np.array([0.0, 1e24, 1.0, 0.0, 1e37, 1e-18, 1e24, 0.0, 1.0, 1e37, 0.0])[:, None]    # of each page's values
    nats = np.array([0.0, -10, 0, 3, -20, 30, -11, 1, -1, -21, 0])                              # and of its scores
    for turn in (0, 4, 7):
        c = Cache(28, 1, 12, 1, page, d)
        g, t = np.roll(grade, turn).repeat(page)[:L], np.roll(nats, turn).repeat(page)[:L]
        k, v = rand(1, L, 1, d, dtype="fp32"), rand(2, L, 1, d, dtype="fp32")
        v *= torch.from_numpy(g.astype(np.float32)).cuda()[:, None, None]
        q = rand(3, nq, G, d, dtype="fp32")
        if tilt:
            k[:, 0, 0] = torch.from_numpy(t.astype(np.float32)).cuda()
            q[..., 0] = d ** 0.5
        else:
            q[0] = 0                                                           # equal scores: an average over all keys
        c.append(k, v, [0], [0, L])
        q = q.bfloat16()
        out, o32 = attend(c, q, [L], [0, nq], 0, max_kv=max_kv)
        pages, scales = [x.cpu().numpy() for x in c.g[:2]], [x.cpu().numpy() for x in c.g[2:4]]
        kk, vv = (dense_cache(pages[i], scales[i], c.table, 0, L)[:, 0] for i in range(2))
        vs = scales[1].astype(np.float64)[c.table[0, np.arange(L) // page], 0]
        x = np.einsum("nhd,ld->nhl", np64(q), kk) * d ** -0.5
        s = (np.einsum("nhd,ld->nhl", np.abs(np64(q)), np.abs(kk)) * d ** -0.5).max(-1, keepdims=True)
        p = np.exp(x - x.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        p_err = 2 * ((d + 8) * U * s + 4 * U) + 300 * U
        bound = (p @ np.abs(vv)) * (2.0 ** -11 + 2 * p_err + 2 * (L / 16 + 64) * 2 * U)
        bound = bound + L * 2.0 ** -32 * 448 * (p * vs).max(-1, keepdims=True)
        near(np64(o32), p @ vv, bound, f"out32, turn {turn}")
        near(np64(out), p @ vv, bound * 1.01 + half_step(p @ vv, q.dtype) * 1.01, f"out, turn {turn}")


@pytest.mark.parametrize("nq", [1, 70])
def test_attention_does_not_see_what_is_masked(nq):
    """NaN scales of pages behind the length, NaN codes behind the last key, and a marked page that no row sees."""
    d, page, L = 128, 64, 330
    c = filled(23, 1, [L], 2, page, d)
    q = rand(4, nq, 4, d)
    ref = check_attention(c, q, [L], [0, nq], 1)
    for i in (0, 1):
        c.g[i][c.table[0, 5], :, L % page:] = 0x7F
        c.g[i + 2][c.table[0, 6:].tolist()] = float("nan")
    assert torch.equal(attend(c, q, [L], [0, nq], 1)[0], ref)
    # a marked page: rows that see any key of it are NaN, the others are as before (token-causal: rows before it)
    c.g[2][c.table[0, 5]] = float("nan")
    got = attend(c, q, [L], [0, nq], 1)[0]
    first = max(0, 320 - (L - nq))                                             # row whose own key is 320
    assert got[first:].isnan().all()
    near(np64(got[:first]), np64(ref[:first]), 0)
    c.g[2][c.table[0, 5]] = 1.0
    c.g[3][c.table[0, 5]] = float("nan")
    got = attend(c, q, [L], [0, nq], 1)[0]
    assert got[first:].isnan().all() and torch.equal(got[:first], ref[:first])


@pytest.mark.parametrize("n", [30, 3])
def test_attention_strides_and_out(n):
    c = filled(24, 1, [200], 2, 64, 128)
    qkv = rand(5, n, 8, 128)
    ref = attend(c, qkv[:, :4].contiguous(), [200], [0, n], 1)[0]
    assert torch.equal(attend(c, qkv[:, :4], [200], [0, n], 1)[0], ref)
    planes = qkv[:, :4].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(attend(c, planes, [200], [0, n], 1)[0], ref)
    odd = torch.zeros(n, 4, 131, dtype=torch.bfloat16, device="cuda")
    odd[..., 3:] = qkv[:, :4]
    out = torch.full((n, 4, 136), 5.0, dtype=torch.bfloat16, device="cuda")
    attend(c, odd[..., 3:], [200], [0, n], 1, out=out[..., 4:132])
    own = qkv[:, :4].clone()
    assert attend(c, own, [200], [0, n], 1, out=own)[0] is own and torch.equal(own, ref)      # over its own queries
    assert torch.equal(out[..., 4:132], ref) and (out[..., :4] == 5).all() and (out[..., 132:] == 5).all()


def test_attention_reports_what_does_not_fit():
    from streaming_causal_video_timestep_b200 import _lib
    c = filled(25, 3, [70, 70, 70], 2, 64, 64)
    for nq in (1, 40):
        q = rand(6, 3 * nq, 2, 64)
        cu = [0, nq, 2 * nq, 3 * nq]
        good = attend(c, q, [70] * 3, cu, 1)[0]
        for kv, cu2, max_q in (([70, -1, 70], cu, nq), ([70, 1000, 70], cu, nq), ([70, 70, 70], [0, nq, 4 * nq, 3 * nq], 3 * nq)):
            out = torch.full_like(q, 3.0)
            attend(c, q, kv, cu2, 1, max_q=max_q, max_kv=70, out=out)    # the same split: the same bits
            assert status() == _lib.LA_EDEVICE and status() == _lib.LA_OK
            assert torch.equal(out[:nq], good[:nq]) and (out[nq:2 * nq] == 3).all()
        keep = int(c.g[4][1, 0])
        for bad in (-1, 10 ** 6):
            c.g[4][1, 0] = bad
            out = attend(c, q, [70] * 3, cu, 1)[0]
            assert status() == _lib.LA_EDEVICE and status() == _lib.LA_OK
            assert torch.equal(out[:nq], good[:nq]) and torch.equal(out[2 * nq:], good[2 * nq:]) and out.isfinite().all()
        c.g[4][1, 0] = keep


def test_offsets_past_32_bits():
    """Pages whose codes lie beyond 4 GiB of the cache, and rotary rows beyond 2^31 elements."""
    from streaming_causal_video_timestep_b200 import op_attention_cache_fp8, op_cache_append_fp8, op_rope_axes
    H, page, d, L = 8, 128, 128, 300
    num = (1 << 32) // (H * page * d) + 40
    big = [torch.empty((num, H, page, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones((num, H), device="cuda") for _ in range(2)]
    table = i32([[num - 1, num - 7, num - 20]])
    small = Cache(41, 1, 3, H, page, d, spare=0)
    k, v = rand(42, L, H, d), rand(43, L, H, d)
    small.append(k, v, [0], [0, L])
    op_cache_append_fp8(k, v, *big, *scales, table, i32([0]), i32([0, L]), L)
    for j in range(3):
        rows = min(page, L - j * page)
        for a, b in zip(big, small.g[:2]):
            assert torch.equal(a[table[0, j]][:, :rows], b[small.table[0, j]][:, :rows])
    for n in (1, 200):
        q = rand(44, n, H, d)
        args = i32([L]), i32([0, n]), n, L
        assert torch.equal(op_attention_cache_fp8(q, *big, *scales, table, *args, causal_block=1),
                           op_attention_cache_fp8(q, *small.g, *args, causal_block=1))
    del big
    T, H = (1 << 31) // (64 * 128) + 5, 64
    x = torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda")
    x[-3:] = rand(45, 3, H, d)
    pos = torch.zeros(T, 3, dtype=torch.int32, device="cuda")
    pos[-3:] = i32([[5, 6, 7], [8, 9, 10], [11, 12, 13]])
    y = op_rope_axes(x, pos, PAIRS[d])
    assert torch.equal(y[-3:], op_rope_axes(x[-3:].clone(), pos[-3:].clone(), PAIRS[d])) and not y[:-3].any()


# ---- together ----------------------------------------------------------------------------------------
def test_stream_of_blocks_and_tokens():
    """Rotate q, append k and v, attend -- a latent block, then single tokens, then a ragged piece, on two streams of
    different length; each attention against the oracle on the cache as it stands."""
    from streaming_causal_video_timestep_b200 import op_rope_axes
    H, G, d, page, B = 2, 2, 128, 64, 2
    c = Cache(40, B, 8, H, page, d)
    lens, seed = np.array([0, 0]), 100
    for new in ([180, 60], [1, 1], [1, 1], [60, 180], [1, 0], [33, 1]):
        cu = np.concatenate([[0], np.cumsum(new)])
        at = np.concatenate([lens[b] + np.arange(new[b]) for b in range(B)])
        pos = np.stack([at // 60 * 7 + 30000, at % 60 // 10, at % 10], 1)
        qkv = rand(seed, cu[-1], H * G + 2 * H, d)
        seed += 1
        c.append(qkv[:, H * G:H * G + H], qkv[:, H * G + H:], lens, cu, pos=pos, pairs=PAIRS[d])
        c.k, c.ks = c.g[0].cpu().numpy().copy(), c.g[2].cpu().numpy().astype(np.float64)   # a K on a rounding border may differ
        c.check_v()
        q = op_rope_axes(qkv[:, :H * G], i32(pos), PAIRS[d])
        lens = lens + np.array(new)
        check_attention(c, q, list(lens), cu, causal=60 if new[0] > 1 else 1)


def test_on_another_stream_and_captured_twice():
    """The three calls on a side stream, and captured into two graphs whose replays overlap on two streams."""
    from streaming_causal_video_timestep_b200 import op_attention_cache_fp8, op_cache_append_fp8, op_rope_axes
    H, d, L = 2, 128, 3000
    kv, cu = i32([L]), i32([0, 1])
    lens, pos = i32([L - 1]), i32([[L // 60, 3, 4]])
    sets = []
    for i in range(2):
        c = filled(50 + i, 1, [L - 1], H, 64, d)
        sets.append((c, rand(60 + i, 1, 3 * H, d)))

    def step(c, qkv):
        q = op_rope_axes(qkv[:, :H], pos, PAIRS[d])
        op_cache_append_fp8(qkv[:, H:2 * H], qkv[:, 2 * H:], *c.g, lens, cu, 1, pos=pos, pairs=PAIRS[d])
        return op_attention_cache_fp8(q, *c.g, kv, cu, 1, L, causal_block=1)

    ref = [step(*s).clone() for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(*sets[0])
    side.synchronize()
    assert torch.equal(got, ref[0])
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, r in zip(outs, ref):
        assert torch.equal(o, r)


def test_stream_argument_and_device_checks():
    from streaming_causal_video_timestep_b200 import op_attention_cache_fp8, op_rope_axes
    x, pos = rand(0, 4, 2, 64), i32(np.arange(12).reshape(4, 3))
    ref = op_rope_axes(x, pos, PAIRS[64])
    c, q, kv, cu = filled(60, 1, [3000], 2, 64, 64), rand(61, 1, 2, 64), i32([3000]), i32([0, 1])
    want = op_attention_cache_fp8(q, *c.g, kv, cu, 1, 3000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(x)
    op_rope_axes(x, pos, PAIRS[64], out=out, stream=side)
    made = op_rope_axes(x, pos, PAIRS[64], stream=side)
    got = op_attention_cache_fp8(q, *c.g, kv, cu, 1, 3000, stream=side)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(made, ref) and torch.equal(got, want)


def test_microbenchmarks_run(monkeypatch):
    from streaming_causal_video_timestep_b200 import microbench
    monkeypatch.setattr(microbench, "_time", lambda fn, iters: (fn(), torch.cuda.synchronize(), 1.0)[2])
    for f in (microbench.bench_rope_axes, microbench.bench_cache_append, microbench.bench_attn_cache,
              microbench.bench_attn_cache_token):
        r = f(1)
        assert r["mode"] and (r.get("bytes") or r.get("flops")) > 0
