"""The expert products and their gradients against a plain 64-bit statement.

Tolerances.  A bf16 output is the float32 sum rounded once: half a step is
2^-8 relative to the next power of two below, i.e. at most 2^-8 |want|.  The
float32 sum of n products of bf16 values (each product exact in float32) is off
by at most n 2^-23 sum|products| even where every addition truncates, so a
result is held to 2^-8 |want| + n 2^-23 S with S the sum of the products'
magnitudes.  Small-integer inputs have exact sums below 2^24, so their results
are held bit for bit."""
import numpy as np
import pytest
import torch

import combine_warp_top_router_b200 as md

from _util import DEV

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def groups(counts, seed=0, gap=0, rows=None):
    """Offsets of experts laid out in a random order, `gap` rows of nobody after each."""
    E = len(counts)
    order = np.random.default_rng(seed).permutation(E)
    off, at = np.zeros(E + 1, dtype=np.int64), 0
    for e in order:
        off[e] = at
        at += counts[e] + gap
    off[E] = at
    rows = at if rows is None else rows
    t = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)  # noqa: E731
    return t(off), t(counts), max(rows, 1), [(e, int(off[e]), int(c)) for e, c in enumerate(counts) if c]


def randn(seed, *shape, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def ints(seed, *shape, hi=4):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(-hi, hi + 1, shape, generator=g, device=DEV).to(torch.bfloat16)


def products64(x, w, spans, nk=True):
    """(products, sums of magnitudes) in 64 bits; rows of nobody are NaN."""
    N = w.shape[1] if nk else w.shape[2]
    y = torch.full((x.shape[0], N), float("nan"), dtype=torch.float64, device=DEV)
    s = torch.zeros_like(y)
    for e, o, c in spans:
        m = w[e].double()
        m = m.t() if nk else m
        y[o:o + c] = x[o:o + c].double() @ m
        s[o:o + c] = x[o:o + c].double().abs() @ m.abs()
    return y, s


def close(got, want, mags, n, mine=None):
    tol = HALF[got.dtype] * want.abs() + n * 2.0 ** -23 * mags + 1e-38
    bad = (got.double() - want).abs() > tol
    if mine is not None:
        bad &= mine[:, None]
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} off, worst " \
        f"{float(((got.double() - want).abs() / tol)[bad].max())} times the tolerance"


def owned(rows, spans):
    m = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for _, o, c in spans:
        m[o:o + c] = True
    return m


SHAPES = [
    # counts, K, N: one token, empty experts, one-row experts, tiles that end at and one past a
    # tile, K and N below, at and past a tile, odd multiples of 8
    ([1], 64, 128), ([1], 8, 8), ([0, 3, 0, 1], 72, 136), ([16, 17, 15, 0, 64, 65], 128, 256),
    ([5] * 40, 2048, 128), ([0] * 63 + [1], 264, 40), ([300, 0, 257, 256, 1, 255], 512, 392),
    ([1000, 13], 1032, 520), ([513], 64, 64), ([2, 1, 700], 200, 1416), ([129] * 9, 192, 1152),
]


@pytest.mark.parametrize("layout", [md.MD_W_NK, md.MD_W_KN])
@pytest.mark.parametrize("counts,K,N", SHAPES)
def test_gemm(counts, K, N, layout):
    off, cnt, rows, spans = groups(counts, seed=K)
    nk = layout == md.MD_W_NK
    E = len(counts)
    x = randn(1, rows, K)
    w = randn(2, *((E, N, K) if nk else (E, K, N)))
    st = md.new_status(DEV)
    y = md.md_expert_gemm(x, w, off, cnt, layout, dev_status=st)
    md.check_status(st)
    want, mags = products64(x, w, spans, nk)
    close(y, want, mags, K, owned(rows, spans))


@pytest.mark.parametrize("op", ["nk", "kn", "gated"])
@pytest.mark.parametrize("counts,K,N", [
    ([500] + [0] * 62 + [3], 200, 136),      # the few-row form with several tiles to an expert
    ([1, 0, 2], 2056, 264),                  # a contraction shared by four CTAs, its blocks uneven
    ([0, 64, 1, 0], 1000, 136), ([40] * 8, 1032, 256),
    ([1] * 200 + [0] * 823 + [7], 72, 64),   # as many experts as there may be
    ([90] * 7 + [0] * 1017, 64, 72), ([300] * 80, 64, 1032)])
def test_forms_are_exact_on_small_integers(counts, K, N, op):
    off, cnt, rows, spans = groups(counts, seed=6, gap=1)
    E, mine, nk = len(counts), None, op != "kn"
    mine = owned(rows, spans)
    st = md.new_status(DEV)
    x = ints(1, rows, K, hi=1)
    if op == "gated":
        w = ints(2, E, 2 * N, K, hi=1)
        act, codes, scales = md.md_expert_gated(x, w, off, cnt, keep=True, dev_status=st)
        md.check_status(st)
        h, _ = products64(x, w, spans)
        g, u = h.chunk(2, 1)
        want = g * torch.sigmoid(g) * u
        # exact sums; the activation's float32 steps (8 * 2^-23) and one rounding
        tol = (2.0 ** -8 + 8 * 2.0 ** -23) * want.abs() + 1e-37
        assert not bool((((act.double() - want).abs() > tol) & mine[:, None]).any())
        for have, true in zip(restore64(codes, scales, N), (g, u)):
            stored, _ = stored64(true[mine])
            assert torch.equal(have[mine], stored)
        return
    w = ints(2, *((E, N, K) if nk else (E, K, N)), hi=1)
    y = md.md_expert_gemm(x, w, off, cnt, md.MD_W_NK if nk else md.MD_W_KN, dev_status=st)
    md.check_status(st)
    want, _ = products64(x, w, spans, nk)
    assert torch.equal(y[mine], want[mine].to(torch.bfloat16))


def test_wgrad_with_the_most_experts():
    counts = [1] * 200 + [0] * 823 + [130]
    off, cnt, rows, spans = groups(counts, seed=2)
    dy, x = ints(1, rows, 72), ints(2, rows, 40)
    dw = md.md_expert_wgrad(dy, x, off, cnt)
    want = torch.zeros(1024, 72, 40, dtype=torch.float64, device=DEV)
    for e, o, c in spans:
        want[e] = dy[o:o + c].double().t() @ x[o:o + c].double()
    assert torch.equal(dw.double(), want)


def test_gradients_are_the_products_differences():
    """The products are linear: <dy, x (w + d)^T - x w^T> = <dw, d> and <dy, (x + d) w^T - x w^T> =
    <dx, d>, exactly on small integers (all sums below 2^24, the outputs below 2^8)."""
    counts, K, N = [33, 0, 70, 5], 64, 72
    off, cnt, rows, _ = groups(counts)
    x, w, dy = ints(1, rows, K, hi=1), ints(2, 4, N, K, hi=1), ints(3, rows, N, hi=1)
    y = md.md_expert_gemm(x, w, off, cnt).double()
    for seed in (4, 5):
        d = (ints(seed, 4, N, K, hi=1) * (torch.rand(4, N, K, device=DEV) < 0.05)).to(torch.bfloat16)
        step = md.md_expert_gemm(x, w + d, off, cnt).double() - y
        dw = md.md_expert_wgrad(dy, x, off, cnt).double()
        assert float((dy.double() * step).sum()) == float((dw * d.double()).sum())
        d = (ints(seed, rows, K, hi=1) * (torch.rand(rows, K, device=DEV) < 0.05)).to(torch.bfloat16)
        step = md.md_expert_gemm(x + d, w, off, cnt).double() - y
        dx = md.md_expert_gemm(dy, w, off, cnt, md.MD_W_KN).double()
        assert float((dy.double() * step).sum()) == float((dx * d.double()).sum())


# ------------------------------------------------------------------ offsets past 32 bits

def _far(rows, counts):
    """Two experts, the second at the very end of `rows`."""
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return t([0, rows - counts[1], rows]), t(counts)


def test_far_rows_of_x_and_y():
    rows, wide, c = 270000, 8192, 90
    off, cnt = _far(rows, [c, c])
    last = slice(rows - c, rows)
    x = torch.zeros(rows, wide, dtype=torch.bfloat16, device=DEV)  # 2.2e9 elements
    x[last] = ints(1, c, wide, hi=1)
    w = ints(2, 2, 64, wide, hi=1)
    y = md.md_expert_gemm(x, w, off, cnt)
    assert torch.equal(y[last], (x[last].double() @ w[1].double().t()).to(torch.bfloat16))
    dy = ints(3, rows, 64, hi=1)
    dw = md.md_expert_wgrad(dy, x, off, cnt)
    assert torch.equal(dw[1].double(), dy[last].double().t() @ x[last].double())
    out = md.md_expert_gemm(dy, w, off, cnt, md.MD_W_KN, out=x)  # [rows, 8192] out
    assert torch.equal(out[last], (dy[last].double() @ w[1].double()).to(torch.bfloat16))


def test_far_experts_of_w_and_dw():
    E, N, K, c = 257, 4096, 2056, 3  # 2.2e9 weights
    counts = [0] * E
    counts[E - 1] = c
    off, cnt, rows, spans = groups(counts)
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device=DEV)
    w[E - 1] = ints(1, N, K, hi=1)
    x = ints(2, rows, K, hi=1)
    y = md.md_expert_gemm(x, w, off, cnt)
    assert torch.equal(y, (x.double() @ w[E - 1].double().t()).to(torch.bfloat16))
    dw = md.md_expert_wgrad(y, x, off, cnt, dw=w)  # bf16
    assert torch.equal(dw[E - 1], (y.double().t() @ x.double()).to(torch.bfloat16))
    assert not bool(dw[:E - 1].any())


def test_far_rows_of_the_checkpoint():
    rows, F, K, c = 140000, 8192, 64, 70
    off, cnt = _far(rows, [c, c])
    last = slice(rows - c, rows)
    x, w = ints(1, rows, K, hi=1), ints(2, 2, 2 * F, K, hi=1)
    act, codes, scales = md.md_expert_gated(x, w, off, cnt, keep=True)  # 2.3e9 codes
    h = x[last].double() @ w[1].double().t()
    want = h[:, :F] * torch.sigmoid(h[:, :F]) * h[:, F:]
    assert bool(((act[last].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want.abs() + 1e-37).all())
    g, u = restore64(codes[last], scales[last], F)
    assert torch.equal(g, stored64(h[:, :F])[0]) and torch.equal(u, stored64(h[:, F:])[0])
    codes[:rows - c].zero_()
    scales[:rows - c].zero_()
    da = torch.zeros(rows, F, dtype=torch.bfloat16, device=DEV)
    da[last] = randn(3, c, F)
    dh, again = md.md_expert_gated_backward(da, codes, scales)
    near = md.md_expert_gated_backward(da[last].contiguous(), codes[last].contiguous(), scales[last].contiguous())
    assert torch.equal(dh[last], near[0]) and torch.equal(again[last], near[1])


def test_far_rows_of_combine_backward():
    T, H, rows = 40, 8192, 270000
    dout = randn(1, T, H)
    y = torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV)
    at = torch.arange(rows - 2 * T, rows, dtype=torch.int32, device=DEV).flip(0).view(T, 2).contiguous()
    y[rows - 2 * T:] = randn(2, 2 * T, H)
    w = torch.rand(T, 2, device=DEV)
    dy, dw = md.md_combine_backward(dout, at, w, y)
    near = md.md_combine_backward(dout, (at - (rows - 2 * T)).contiguous(), w, y[rows - 2 * T:].contiguous())
    assert torch.equal(dy[rows - 2 * T:], near[0]) and torch.equal(dw, near[1])


@pytest.mark.parametrize("layout", [md.MD_W_NK, md.MD_W_KN])
@pytest.mark.parametrize("counts,K,N", [([7, 0, 33], 128, 136), ([260, 31, 0, 512], 320, 264)])
def test_gemm_is_exact_on_small_integers_and_leaves_other_rows(counts, K, N, layout):
    off, cnt, rows, spans = groups(counts, seed=3, gap=5)
    nk = layout == md.MD_W_NK
    x = ints(1, rows, K)
    w = ints(2, *((len(counts), N, K) if nk else (len(counts), K, N)), hi=1)
    mine = owned(rows, spans)
    x[~mine] = float("nan")  # rows of nobody are not read into a result
    y = torch.full((rows, N), 77.0, dtype=torch.bfloat16, device=DEV)
    md.md_expert_gemm(x, w, off, cnt, layout, out=y)
    want, _ = products64(x, w, spans, nk)
    assert torch.equal(y[mine], want[mine].to(torch.bfloat16))
    assert bool((y[~mine] == 77.0).all())


def test_gemm_keeps_nan_and_inf_to_their_row_and_expert():
    counts, K, N = [3, 5, 300, 4], 136, 200
    off, cnt, rows, spans = groups(counts, seed=1)
    x, w = randn(1, rows, K), randn(2, 4, N, K)
    base = md.md_expert_gemm(x, w, off, cnt)
    r = int(off[2]) + 299
    x[r, K - 1] = float("inf")
    w[0, N - 1, K - 1] = float("nan")
    y = md.md_expert_gemm(x, w, off, cnt)
    same = torch.ones_like(y, dtype=torch.bool)
    same[r] = False
    same[int(off[0]):int(off[0]) + 3, N - 1] = False
    assert torch.equal(y[same], base[same])
    assert not bool(torch.isfinite(y[r]).any())
    assert bool(torch.isnan(y[int(off[0]):int(off[0]) + 3, N - 1]).all())
    # the contraction's tail (K is no multiple of a block) must not meet the next expert's weights
    wk = randn(3, 4, K, N)
    kn = md.md_expert_gemm(x, wk, off, cnt, md.MD_W_KN)
    wk2 = wk.clone()
    wk2[1] = float("nan")
    again = md.md_expert_gemm(x, wk2, off, cnt, md.MD_W_KN)
    mine = torch.ones(rows, dtype=torch.bool, device=DEV)
    mine[int(off[1]):int(off[1]) + 5] = False
    mine[r] = False
    assert torch.equal(kn[mine], again[mine])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 8, 8), ([0, 3, 0, 1], 136, 72), ([16, 17, 15, 0, 64, 65], 256, 264), ([5] * 40, 128, 512),
    ([300, 0, 257, 256, 1, 255], 392, 520), ([2, 1, 700], 1416, 200), ([63, 64, 65, 127, 129], 128, 1032)])
def test_wgrad(counts, N, K, dtype):
    off, cnt, rows, spans = groups(counts, seed=N, gap=3)
    dy, x = randn(1, rows, N), randn(2, rows, K)
    mine = owned(rows, spans)
    dy[~mine], x[~mine] = float("nan"), float("inf")  # rows of nobody, right behind each expert's last
    st = md.new_status(DEV)
    dw = md.md_expert_wgrad(dy, x, off, cnt, out_dtype=dtype, dev_status=st)
    md.check_status(st)
    assert dw.shape == (len(counts), N, K) and dw.dtype == dtype
    want = torch.zeros(len(counts), N, K, dtype=torch.float64, device=DEV)
    mags = torch.zeros_like(want)
    for e, o, c in spans:
        want[e] = dy[o:o + c].double().t() @ x[o:o + c].double()
        mags[e] = dy[o:o + c].double().abs().t() @ x[o:o + c].double().abs()
    close(dw, want, mags, max(counts))


def test_wgrad_accumulates_and_clears():
    counts, N, K = [70, 0, 33], 136, 264
    off, cnt, rows, spans = groups(counts)
    dy, x = ints(1, rows, N), ints(2, rows, K)
    want = torch.zeros(3, N, K, dtype=torch.float64, device=DEV)
    for e, o, c in spans:
        want[e] = dy[o:o + c].double().t() @ x[o:o + c].double()
    dw = torch.full((3, N, K), 5.0, device=DEV)
    assert md.md_expert_wgrad(dy, x, off, cnt, dw=dw, accumulate=True) is dw
    assert torch.equal(dw.double(), want + 5)
    md.md_expert_wgrad(dy, x, off, cnt, dw=dw)
    assert torch.equal(dw.double(), want)


def test_wgrad_into_a_buffer_of_16_byte_alignment():
    counts, N, K = [70, 0, 33], 136, 264
    off, cnt, rows, spans = groups(counts)
    dy, x = ints(1, rows, N), ints(2, rows, K)
    want = md.md_expert_wgrad(dy, x, off, cnt)
    for shift in (4, 8):
        flat = torch.full((3 * N * K + 16,), 9.0, device=DEV)
        dw = flat[shift:shift + 3 * N * K].view(3, N, K)
        md.md_expert_wgrad(dy, x, off, cnt, dw=dw)
        assert torch.equal(dw, want)
        assert bool((flat[:shift] == 9.0).all()) and bool((flat[shift + 3 * N * K:] == 9.0).all())


@pytest.mark.parametrize("counts", [[2049], [5000, 0, 2048, 100]])
def test_wgrad_of_long_experts(counts):
    """Experts whose rows are summed in several parts, into a fresh and a kept dw."""
    N, K = 264, 520
    off, cnt, rows, spans = groups(counts, seed=5)
    dy, x = ints(1, rows, N, hi=2), ints(2, rows, K, hi=2)
    want = torch.zeros(len(counts), N, K, dtype=torch.float64, device=DEV)
    for e, o, c in spans:
        want[e] = dy[o:o + c].double().t() @ x[o:o + c].double()
    dw = md.md_expert_wgrad(dy, x, off, cnt)
    assert torch.equal(dw.double(), want)
    md.md_expert_wgrad(dy, x, off, cnt, dw=dw, accumulate=True)
    assert torch.equal(dw.double(), 2 * want)
    assert torch.equal(md.md_expert_wgrad(dy, x, off, cnt, out_dtype=torch.bfloat16), want.to(torch.bfloat16))


@pytest.mark.parametrize("hi", [1, 16, 63, 64, 130])
def test_wgrad_of_many_short_experts(hi):
    """Tiles of one to three blocks, so that the loads run several tiles ahead."""
    E, N, K = 96, 1032, 264
    counts = np.random.default_rng(hi).integers(1, hi + 1, E).tolist()
    off, cnt, rows, spans = groups(counts, seed=hi, gap=1)
    dy, x = ints(1, rows, N, hi=2), ints(2, rows, K, hi=2)
    mine = owned(rows, spans)
    dy[~mine], x[~mine] = float("nan"), float("nan")
    st = md.new_status(DEV)
    dw = md.md_expert_wgrad(dy, x, off, cnt, dev_status=st)
    md.check_status(st)
    for e, o, c in spans:
        assert torch.equal(dw[e].double(), dy[o:o + c].double().t() @ x[o:o + c].double())


@pytest.mark.parametrize("op", ["nk", "kn", "gated", "wgrad"])
def test_many_tiles_of_two_products(op):
    """Enough tiles that each takes 512 weight rows, some of whose second halves are partly or
    wholly outside; skewed counts."""
    counts = [0, 700, 1, 256, 257, 513, 90, 33, 1200, 0, 64, 300, 129, 511, 512, 31]
    K, N = 328, 1416
    off, cnt, rows, spans = groups(counts, seed=8, gap=1)
    E = len(counts)
    x = ints(1, rows, K, hi=2)
    if op == "wgrad":
        dy = ints(2, rows, N, hi=2)
        want = torch.zeros(E, N, K, dtype=torch.float64, device=DEV)
        for e, o, c in spans:
            want[e] = dy[o:o + c].double().t() @ x[o:o + c].double()
        assert torch.equal(md.md_expert_wgrad(dy, x, off, cnt).double(), want)
        return
    mine = owned(rows, spans)
    if op == "gated":
        w = randn(2, E, 2 * N, K, scale=1.5 / 16)
        got = md.md_expert_gated(x, w, off, cnt)
        h, mags = products64(x, w, spans)
        g, u = h.chunk(2, 1)
        mg, mu = mags.chunk(2, 1)
        want = g * torch.sigmoid(g) * u
        tol = 2.0 ** -8 * want.abs() + K * 2.0 ** -23 * (1.1 * mg * u.abs() + mu * g.abs()) * 1.01 \
            + 8 * 2.0 ** -23 * want.abs() + 1e-37
        bad = ((got.double() - want).abs() > tol) & mine[:, None]
        assert not bool(bad.any()), int(bad.sum())
        return
    nk = op == "nk"
    w = ints(2, *((E, N, K) if nk else (E, K, N)), hi=1)
    y = md.md_expert_gemm(x, w, off, cnt, md.MD_W_NK if nk else md.MD_W_KN)
    want, _ = products64(x, w, spans, nk)
    assert torch.equal(y[mine], want[mine].to(torch.bfloat16))


# ------------------------------------------------------------------ gated, checkpoint

def stored64(h):
    """What an 8-bit checkpoint of h (float64) holds, and the scales' bytes."""
    out, codes = torch.empty_like(h), []
    for c in range(0, h.shape[1], 32):
        b = h[:, c:c + 32]
        top = torch.where(torch.isfinite(b), b.abs(), torch.zeros_like(b)).amax(1, keepdim=True)
        s = torch.full_like(top, -127.0)
        for e in range(-127, 121):  # the smallest scale that holds the block
            s = torch.where(448 * 2.0 ** e < top, torch.full_like(top, e + 1.0), s)
        v = b / torch.exp2(s)
        mag = torch.where(torch.isfinite(v), v.abs(), torch.ones_like(v)).clamp(min=2.0 ** -6)
        step = torch.exp2(torch.floor(torch.log2(mag)) - 3)
        q = torch.round(v / step) * step * torch.exp2(s)
        out[:, c:c + 32] = torch.where(torch.isfinite(b), q, torch.full_like(b, float("nan")))
        codes.append((s + 127).to(torch.uint8))
    return out, torch.cat(codes, 1)


def restore64(codes, scales, F):
    B = scales.shape[1] // 2
    at = torch.arange(F, device=DEV) // 32
    sg, su = scales[:, :B][:, at].double() - 127, scales[:, B:][:, at].double() - 127
    return codes[:, :F].double() * torch.exp2(sg), codes[:, F:].double() * torch.exp2(su)


GATED = [([1], 8, 8), ([3, 0, 1], 64, 64), ([17] * 5, 136, 72), ([0, 40, 2], 2048, 128), ([300, 1, 0, 257], 264, 200),
         ([129, 511], 512, 456)]


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("counts,K,F", GATED)
def test_gated(counts, K, F, keep):
    off, cnt, rows, spans = groups(counts, seed=F, gap=2)
    x, w = randn(1, rows, K), randn(2, len(counts), 2 * F, K, scale=1.5 * K ** -0.5)
    mine = owned(rows, spans)
    st = md.new_status(DEV)
    got = md.md_expert_gated(x, w, off, cnt, keep=keep, dev_status=st)
    md.check_status(st)
    a = got[0] if keep else got
    h, mags = products64(x, w, spans)
    g, u = h.chunk(2, 1)
    mg, mu = mags.chunk(2, 1)
    s = torch.sigmoid(g)
    want = g * s * u
    # the sums' error through the activation (|d silu| <= 1.1, |silu(g)| <= |g|), and float32's exp,
    # division and products: expf is within 2 ulp, the rest 1/2 each -- 8 * 2^-23 covers them; expf's
    # error reaches silu at most times 1, since s(1 - s) |exp'| / s <= 1
    tol = 2.0 ** -8 * want.abs() + K * 2.0 ** -23 * (1.1 * mg * u.abs() + mu * g.abs()) * 1.01 \
        + 8 * 2.0 ** -23 * want.abs() + 1e-37
    bad = ((a.double() - want).abs() > tol) & mine[:, None]
    assert not bool(bad.any()), int(bad.sum())
    if keep:
        _, codes, scales = got
        rg, ru = restore64(codes, scales, F)
        for have, true, m in ((rg, g, mg), (ru, u, mu)):
            err = K * 2.0 ** -23 * m
            # half a step of e4m3: 2^-4 of the value, or 2^-10 of the scale; the scale is at most
            # twice the smallest one that the block's largest value needs
            top = torch.nn.functional.pad(true.abs(), (0, -F % 32)).view(rows, -1, 32).amax(-1)
            top = top.repeat_interleave(32, 1)[:, :F]
            lim = 2.0 ** -4 * (true.abs() + err) + 2.0 ** -10 * 2 * (top + err) / 448 + err
            bad = ((have - true).abs() > lim) & mine[:, None]
            assert not bool(bad.any()), int(bad.sum())


@pytest.mark.parametrize("counts,F", [([5, 0, 2], 40), ([300, 20], 96)])
def test_checkpoint_is_exact_where_the_sums_are(counts, F):
    """One-hot rows pick a weight column, so g and u are bf16 values chosen here: scales and codes
    must be the definition's to the bit, at powers of two, at 448's edge, with zeros and tiny values."""
    K = 64
    off, cnt, rows, spans = groups(counts, seed=2)
    E = len(counts)
    g = torch.Generator().manual_seed(4)
    v = torch.randn(E, 2 * F, K, generator=g) * torch.exp2(torch.randint(-30, 30, (E, 2 * F, K), generator=g).float())
    edge = torch.tensor([448.0, 450.0, 447.0, 449.0, 1.75, 1.7578125, 256.0, 2.0 ** -120, 2.0 ** -126, 2.0 ** 100, 0.0, -0.0,
                         1.0, 2.0 ** -10, 464.0, 0.0])
    v[:, :, :16] = edge * torch.where(torch.rand(E, 2 * F, 16, generator=g) < 0.5, -1.0, 1.0)
    v[:, :, 16] = 0
    v[:, 1, 17] = 448.0
    v[:, 0, 17] = 450.0
    w = v.to(torch.bfloat16).to(DEV)
    pick = torch.randint(0, K, (rows,), generator=g).to(DEV)
    pick[: min(rows, 18)] = torch.arange(min(rows, 18), device=DEV)
    x = torch.nn.functional.one_hot(pick, K).to(torch.bfloat16)
    act, codes, scales = md.md_expert_gated(x, w, off, cnt, keep=True)
    for e, o, c in spans:
        h = w[e][:, pick[o:o + c]].t().double()
        for half, at in ((h[:, :F], 0), (h[:, F:], 1)):
            want, sc = stored64(half)
            B = scales.shape[1] // 2
            assert torch.equal(scales[o:o + c, at * B:(at + 1) * B], sc)
            have = restore64(codes, scales, F)[at][o:o + c]
            assert torch.equal(have, want)


def test_checkpoint_stores_inf_and_nan_as_nan():
    K, F = 64, 40
    off, cnt, rows, _ = groups([4])
    w = randn(5, 1, 2 * F, K)
    x = torch.nn.functional.one_hot(torch.arange(4, device=DEV), K).to(torch.bfloat16)
    x = torch.where(x > 0, x, torch.zeros_like(x))
    clean = md.md_expert_gated(x, w, off, cnt, keep=True)
    big = w.clone()
    big[0, 3, 1] = 3.0e38
    x[1, 1] = 3.0e38  # 9e76: Inf in float32, in one value of row 1
    big[0, torch.arange(2 * F) != 3, 1] = 0
    act, codes, scales = md.md_expert_gated(x, big, off, cnt, keep=True)
    g, u = restore64(codes, scales, F)
    assert bool(torch.isnan(g[1, 3])) and int(torch.isnan(g).sum()) == 1 and not bool(torch.isnan(u).any())
    for r in (0, 2, 3):
        assert torch.equal(codes[r].view(torch.uint8), clean[1][r].view(torch.uint8))
    dh, again = md.md_expert_gated_backward(torch.ones(4, F, dtype=torch.bfloat16, device=DEV), codes, scales)
    assert bool(torch.isnan(dh[1, 3])) and bool(torch.isnan(again[1, 3]))
    assert int(torch.isnan(again).sum()) == 1


@pytest.mark.parametrize("rows,F", [(1, 8), (3, 40), (257, 72), (64, 1416), (1000, 256)])
def test_gated_backward(rows, F):
    g = torch.Generator(device=DEV).manual_seed(rows)
    B = -(-F // 32)
    codes = torch.randint(0, 256, (rows, 2 * F), generator=g, device=DEV, dtype=torch.uint8)
    codes[(codes & 0x7f) == 0x7f] = 0x30  # NaN codes apart
    codes = codes.view(torch.float8_e4m3fn)
    scales = torch.randint(112, 122, (rows, 2 * B), generator=g, device=DEV, dtype=torch.uint8)
    scales[0, 0] = 0
    da = randn(2, rows, F)
    dh, act = md.md_expert_gated_backward(da, codes, scales)
    G, U = restore64(codes, scales, F)
    d, s = da.double(), torch.sigmoid(G)
    dg, du, a = d * U * (s + G * s * (1 - s)), d * G * s, G * s * U
    # float32: s has a relative error below 4 ulp, so does each product; 1 + x (1 - s) cancels where
    # x (1 - s) is near -1 and its terms reach |x| (1 - s), so dg is held to its terms' magnitudes;
    # 1 - s is off by 2^-24 of s's size whatever its own, hence the term |x| s without (1 - s)
    tiny = 2.0 ** -133  # bf16's last step below its normal range, and float32's products there
    lim = lambda want, terms: 2.0 ** -8 * want.abs() + 16 * 2.0 ** -24 * terms + tiny  # noqa: E731
    assert bool(((dh[:, :F].double() - dg).abs() <= lim(dg, (d * U).abs() * s * (1 + G.abs()))).all())
    assert bool(((dh[:, F:].double() - du).abs() <= lim(du, du.abs())).all())
    assert bool(((act.double() - a).abs() <= lim(a, a.abs())).all())
    dh2, none = md.md_expert_gated_backward(da, codes, scales, want_act=False)
    assert none is None and torch.equal(dh2, dh)


def test_gated_backward_against_differences():
    """The formula is the derivative of the forward's: central differences in 64 bits."""
    rows, F = 6, 32
    g = torch.Generator(device=DEV).manual_seed(9)
    codes = (torch.randn(rows, 2 * F, generator=g, device=DEV) * 2).to(torch.float8_e4m3fn)
    scales = torch.full((rows, 2), 127, dtype=torch.uint8, device=DEV)
    da = randn(3, rows, F)
    dh, _ = md.md_expert_gated_backward(da, codes, scales)
    G, U = restore64(codes, scales, F)
    f = lambda p, q: (p * torch.sigmoid(p) * q * da.double())  # noqa: E731
    h = 1e-5  # error h^2 |f'''| / 6 <= 1e-10 |da u|, far below a bf16 step of the terms
    dg, du = (f(G + h, U) - f(G - h, U)) / (2 * h), (f(G, U + h) - f(G, U - h)) / (2 * h)
    size = (da.double() * U).abs() + (da.double() * G).abs()
    assert bool(((dh[:, :F].double() - dg).abs() <= 2.0 ** -8 * dg.abs() + 1e-6 * size + 1e-9).all())
    assert bool(((dh[:, F:].double() - du).abs() <= 2.0 ** -8 * du.abs() + 1e-6 * size + 1e-9).all())


# ------------------------------------------------------------------ combine backward

@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (5, 2, 264), (33, 6, 2048), (64, 8, 1032), (17, 32, 72), (3, 3, 4096)])
def test_combine_backward(T, k, H):
    g = torch.Generator(device=DEV).manual_seed(T)
    rows = T * k + 4
    perm = torch.randperm(rows, generator=g, device=DEV)[:T * k].to(torch.int32).view(T, k)
    dout, y = randn(1, T, H), randn(2, rows, H)
    w = torch.rand(T, k, generator=g, device=DEV)
    dy = torch.full((rows, H), 9.0, dtype=torch.bfloat16, device=DEV)
    st = md.new_status(DEV)
    got, dw = md.md_combine_backward(dout, perm.contiguous(), w, y, dy=dy, dev_status=st)
    md.check_status(st)
    assert got is dy
    flat = perm.flatten().long()
    want = (w[:, :, None] * dout.float()[:, None]).to(torch.bfloat16).view(T * k, H)  # one float32 product, one rounding
    assert torch.equal(dy[flat], want)
    left = torch.ones(rows, dtype=torch.bool, device=DEV)
    left[flat] = False
    assert bool((dy[left] == 9.0).all())
    d64 = (y[flat].double().view(T, k, H) * dout.double()[:, None])
    assert bool(((dw.double() - d64.sum(-1)).abs() <= H * 2.0 ** -24 * d64.abs().sum(-1) + 1e-30).all())
    dy2, none = md.md_combine_backward(dout, perm.contiguous(), w, y_rows=rows)
    assert none is None and torch.equal(dy2[flat], want)


def test_combine_backward_skips_and_reports_bad_rows():
    T, k, H = 4, 2, 64
    rows = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k)
    rows[1, 0], rows[2, 1] = -1, T * k
    dout, y = randn(1, T, H), randn(2, T * k, H)
    w = torch.rand(T, k, device=DEV)
    st = md.new_status(DEV)
    dy = torch.full((T * k, H), 9.0, dtype=torch.bfloat16, device=DEV)
    _, dw = md.md_combine_backward(dout, rows, w, y, dy=dy, dev_status=st)
    assert int(st.item()) == md.MD_ERR_DATA
    assert float(dw[1, 0]) == 0 and float(dw[2, 1]) == 0
    assert bool((dy[2] == 9.0).all()) and bool((dy[5] == 9.0).all())


# ------------------------------------------------------------------ errors, streams, graphs

def test_bad_ranges_are_empty_and_reported():
    E, K, N, rows = 4, 64, 64, 40
    x, w = ints(1, rows, K), ints(2, E, N, K, hi=1)
    cnt = torch.tensor([10, -1, 35, 10], dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 10, 10, -3], dtype=torch.int32, device=DEV)
    st = md.new_status(DEV)
    y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device=DEV)
    md.md_expert_gemm(x, w, off, cnt, out=y, dev_status=st)
    assert int(st.item()) == md.MD_ERR_DATA
    want, _ = products64(x, w, [(0, 0, 10)])
    assert torch.equal(y[:10], want[:10].to(torch.bfloat16)) and bool((y[10:] == 7.0).all())
    dw = md.md_expert_wgrad(x, x, off, cnt, dev_status=st)
    assert int(st.item()) == md.MD_ERR_DATA
    assert torch.equal(dw[0].double(), x[:10].double().t() @ x[:10].double()) and not bool(dw[1:].any())
    act = torch.full((rows, N // 2), 7.0, dtype=torch.bfloat16, device=DEV)
    md.md_expert_gated(x, w, off, cnt, out=act, dev_status=st)
    assert int(st.item()) == md.MD_ERR_DATA and bool((act[10:] == 7.0).all())


def test_no_rows():
    E, K, N = 3, 64, 72
    x, w = randn(1, 0, K), randn(2, E, N, K)
    z = torch.zeros(E, dtype=torch.int32, device=DEV)
    st = md.new_status(DEV)
    assert md.md_expert_gemm(x, w, z, z, dev_status=st).shape == (0, N)
    with pytest.raises(md.MoeDispatchError):  # F = 36 is no multiple of 8
        md.md_expert_gated(x, w, z, z, keep=True)
    act, codes, scales = md.md_expert_gated(x, randn(2, E, 80, K), z, z, keep=True, dev_status=st)
    assert act.shape == (0, 40) and codes.shape == (0, 80)
    dh, _ = md.md_expert_gated_backward(randn(3, 0, 40), codes, scales)
    assert dh.shape == (0, 80)
    dw = torch.full((E, N, K), 3.0, device=DEV)
    md.md_expert_wgrad(randn(1, 0, N), x, z, z, dw=dw, accumulate=True)
    assert bool((dw == 3.0).all())
    md.md_expert_wgrad(randn(1, 0, N), x, z, z, dw=dw)
    assert not bool(dw.any())
    dy, g = md.md_combine_backward(randn(1, 0, 64), torch.zeros(0, 2, dtype=torch.int32, device=DEV),
                                   torch.zeros(0, 2, device=DEV), randn(1, 0, 64))
    assert dy.shape == (0, 64) and g.shape == (0, 2)
    md.check_status(st)


def test_rows_but_no_expert_has_any():
    E, K, N, rows = 5, 64, 72, 9
    z = torch.zeros(E, dtype=torch.int32, device=DEV)
    y = torch.full((rows, N), 3.0, dtype=torch.bfloat16, device=DEV)
    md.md_expert_gemm(randn(1, rows, K), randn(2, E, N, K), z, z, out=y)
    assert bool((y == 3.0).all())
    assert not bool(md.md_expert_wgrad(randn(1, rows, N), randn(1, rows, K), z, z).any())


def _layer(x, w13, w2, idx, gates, L, dout):
    """One expert layer forward and backward through the library's own calls."""
    rows = idx.numel()
    off, cnt = L.expert_offsets, L.expert_counts
    xs = md.md_dispatch_permute(x, L.assign_row, out_rows=rows)
    act, codes, scales = md.md_expert_gated(xs, w13, off, cnt, keep=True)
    y = md.md_expert_gemm(act, w2, off, cnt)
    out = md.md_combine(y, L.assign_row, idx, gates)
    dy, dgate = md.md_combine_backward(dout, L.assign_row, gates, y)
    da = md.md_expert_gemm(dy, w2, off, cnt, md.MD_W_KN)
    dh, again = md.md_expert_gated_backward(da, codes, scales)
    dw2 = md.md_expert_wgrad(dy, again, off, cnt)
    dw13 = md.md_expert_wgrad(dh, xs, off, cnt)
    dxs = md.md_expert_gemm(dh, w13, off, cnt, md.MD_W_KN)
    dx = md.md_combine(dxs, L.assign_row, idx, torch.ones_like(gates))
    return out, dgate, dw2, dw13, dx


def _layer_inputs(T=192, E=16, k=4, R=4, H=256, F=136, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    idx, gates = md.md_route_topk(torch.randn(T, E, generator=g, device=DEV), k)
    p = torch.randperm(E, generator=g, device=DEV).to(torch.int32) % R
    L = md.md_dispatch_layout(idx, E, R, p.to(torch.int32), md.MD_DEDUP)
    return (randn(seed + 1, T, H), randn(seed + 2, E, 2 * F, H, scale=1.5 * H ** -0.5),
            randn(seed + 3, E, H, F, scale=F ** -0.5), idx, gates, L, randn(seed + 4, T, H, scale=0.1))


def test_a_layer_forward_and_backward_against_autograd_in_64_bits():
    """Dispatch, experts, combine and back, against torch's autograd of the layer in 64 bits.  Each
    tensor on the way is rounded to bf16 (relative 2^-9 rms at most) and the checkpoint to e4m3
    (2^-4 at most, 2^-4/sqrt(3) rms): errors are compared in the 2-norm.  The forward passes five
    roundings: 5 * 2^-8 holds it.  The gradients carry e4m3's error of g and u into da's two factors
    and into a: at most twice 2^-4 relative to their terms, which random signs average; 2^-3 holds
    the weight gradients and dx.  The gates' gradient does not pass the checkpoint: 5 * 2^-8."""
    x, w13, w2, idx, gates, L, dout = _layer_inputs()
    out, dgate, dw2, dw13, dx = _layer(x, w13, w2, idx, gates, L, dout)
    X, W13, W2, G = (t.double().requires_grad_() for t in (x, w13, w2, gates))
    F = w2.shape[2]
    total = torch.zeros_like(X)
    for j in range(idx.shape[1]):
        e = idx[:, j].long()
        h = torch.einsum("th,tnh->tn", X, W13[e])
        a = torch.nn.functional.silu(h[:, :F]) * h[:, F:]
        total = total + G[:, j:j + 1] * torch.einsum("tf,thf->th", a, W2[e])
    total.backward(dout.double())
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert rel(out, total.detach()) < 5 * 2.0 ** -8
    assert rel(dgate, G.grad) < 5 * 2.0 ** -8
    for got, want in ((dw2, W2.grad), (dw13, W13.grad), (dx, X.grad)):
        assert rel(got, want) < 2.0 ** -3


def test_a_layer_is_the_same_every_time_on_another_stream_and_in_a_graph():
    a = _layer_inputs(seed=7)
    want = _layer(*a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = _layer(*a)
    torch.cuda.current_stream().wait_stream(s)
    for u, v in zip(side, want):
        assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _layer(*a)
    other = _layer_inputs(seed=8)
    for dst, src in zip((a[0], a[1], a[2], a[6]), (other[0], other[1], other[2], other[6])):
        dst.copy_(src)
    fresh = _layer(*a)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for u, v in zip(captured, fresh):
        assert torch.equal(u, v)


def test_two_streams_at_once():
    one, two = _layer_inputs(seed=1), _layer_inputs(T=640, F=264, seed=2)
    want = [_layer(*one), _layer(*two)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        with torch.cuda.stream(s1):
            got[0] = _layer(*one)
        with torch.cuda.stream(s2):
            got[1] = _layer(*two)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for u, v in zip(g, w):
            assert torch.equal(u, v)


def test_refusals():
    K, N, E, rows = 64, 72, 3, 10
    x, w = randn(1, rows, K), randn(2, E, N, K)
    off, cnt, _, _ = groups([4, 3, 3])
    with pytest.raises(TypeError):
        md.md_expert_gemm(x.float(), w, off, cnt)
    with pytest.raises(TypeError):
        md.md_expert_gemm(x, w, off.long(), cnt)
    with pytest.raises(ValueError):
        md.md_expert_gemm(x, w.transpose(1, 2), off, cnt)          # not contiguous
    with pytest.raises(ValueError):
        md.md_expert_gemm(x, randn(2, E, N, K + 8), off, cnt)      # another K
    with pytest.raises(ValueError):
        md.md_expert_gemm(x, w, off, cnt[:2].contiguous())         # too few counts
    with pytest.raises(ValueError):
        md.md_expert_gemm(x, w, off, cnt, out=torch.empty(rows, N - 8, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        md.md_expert_gemm(x, w, off, cnt, w_layout=2)
    with pytest.raises(ValueError):
        md.md_expert_gemm(x.cpu(), w, off, cnt)
    for bad_x, bad_w in ((randn(1, rows, 12), randn(2, E, N, 12)), (x, randn(2, E, 12, K))):
        with pytest.raises(md.MoeDispatchError) as err:
            md.md_expert_gemm(bad_x, bad_w, off, cnt)
        assert err.value.code == md.MD_ERR_ARG
    with pytest.raises(md.MoeDispatchError):                        # 16-byte alignment
        md.md_expert_gemm(randn(1, rows * K + 1).view(-1)[1:].view(rows, K), w, off, cnt)
    with pytest.raises(ValueError):
        md.md_expert_gated(x, randn(2, E, 9, K), off, cnt)
    with pytest.raises(ValueError):
        md.md_expert_wgrad(randn(1, rows, N), x, off, cnt, accumulate=True)
    with pytest.raises(ValueError):
        md.md_expert_wgrad(randn(1, rows, N), x, off, cnt, accumulate=True,
                           dw=torch.zeros(E, N, K, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError):
        md.md_expert_wgrad(randn(1, rows, N), x, off, cnt, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        md.md_expert_wgrad(randn(1, rows + 1, N), x, off, cnt)
    with pytest.raises(TypeError):
        md.md_expert_gated_backward(randn(1, 4, 32), torch.zeros(4, 64, dtype=torch.uint8, device=DEV),
                                    torch.zeros(4, 2, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        md.md_expert_gated_backward(randn(1, 4, 32), torch.zeros(4, 64, device=DEV).to(torch.float8_e4m3fn),
                                    torch.zeros(4, 1, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        md.md_combine_backward(randn(1, 4, 64), torch.zeros(4, 2, dtype=torch.int32, device=DEV),
                               torch.zeros(4, 2, device=DEV), dw=torch.zeros(4, 2, device=DEV))


def test_a_wait_that_runs_out_is_reported_and_leaves_the_gpu_usable():
    """With a poll limit of one nearly every wait inside gives up: the kernel must free what it
    holds, report, and the next call must be right."""
    from combine_warp_top_router_b200 import binding
    counts, K, N = [300, 40, 0, 700], 512, 520
    off, cnt, rows, spans = groups(counts)
    x, w = ints(1, rows, K, hi=1), ints(2, 4, N, K, hi=1)
    st = md.new_status(DEV)
    binding.lib().md_set_test_hooks(1, -1, -1)
    try:
        md.md_expert_gemm(x, w, off, cnt, dev_status=st)
        assert int(st.item()) == md.MD_ERR_TIMEOUT
        md.md_expert_wgrad(x, x, off, cnt, dev_status=st)
        assert int(st.item()) == md.MD_ERR_TIMEOUT
    finally:
        binding.lib().md_set_test_hooks(0, -1, -1)
    y = md.md_expert_gemm(x, w, off, cnt, dev_status=st)
    md.check_status(st)
    want, _ = products64(x, w, spans)
    assert torch.equal(y, want.to(torch.bfloat16))


@pytest.mark.parametrize("form", ["wide", "wide gated", "shared"])
def test_a_wait_that_runs_out_in_each_form(form):
    """The same in the pairs' kernel and where CTAs share a contraction."""
    from combine_warp_top_router_b200 import binding
    counts, K, N = ([2], 2048, 264) if form == "shared" else ([300] * 40, 512, 528)
    off, cnt, rows, spans = groups(counts)
    x, w = ints(1, rows, K, hi=1), ints(2, len(counts), N, K, hi=1)

    def call(st):
        if form == "wide gated":
            return md.md_expert_gated(x, w, off, cnt, keep=True, dev_status=st)
        return md.md_expert_gemm(x, w, off, cnt, dev_status=st)

    st = md.new_status(DEV)
    binding.lib().md_set_test_hooks(1, -1, -1)
    try:
        call(st)
        assert int(st.item()) == md.MD_ERR_TIMEOUT
    finally:
        binding.lib().md_set_test_hooks(0, -1, -1)
    first, again = call(st), call(st)
    md.check_status(st)
    for a, b in zip(first, again):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    if form != "wide gated":
        want, _ = products64(x, w, spans)
        assert torch.equal(first, want.to(torch.bfloat16))


@pytest.mark.parametrize("op", ["gemm", "gated", "wgrad"])
def test_first_call_may_be_captured(op):
    """A call whose shapes no warm-up has seen, captured at once and replayed on new inputs."""
    counts, K, N = [70, 0, 300, 5], 200, 144
    off, cnt, rows, spans = groups(counts)
    x, w, dy = ints(1, rows, K, hi=1), ints(2, 4, N, K, hi=1), ints(3, rows, N, hi=1)
    call = {"gemm": lambda: md.md_expert_gemm(x, w, off, cnt),
            "gated": lambda: md.md_expert_gated(x, w, off, cnt, keep=True)[1].view(torch.uint8),
            "wgrad": lambda: md.md_expert_wgrad(dy, x, off, cnt)}[op]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    # other rows, another split of them among the experts
    x.copy_(ints(7, rows, K, hi=1))
    off2, cnt2, _, _ = groups([5, 300, 0, 70], seed=3)
    off.copy_(off2)
    cnt.copy_(cnt2)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, call())


def test_combine_backward_refuses_rows_that_are_not_ys():
    T, k, H = 4, 2, 64
    dout, y = randn(1, T, H), randn(2, T * k, H)
    rows = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k)
    w = torch.rand(T, k, device=DEV)
    for bad in (T * k + 3, T * k - 1):
        with pytest.raises(ValueError):
            md.md_combine_backward(dout, rows, w, y, y_rows=bad)
        with pytest.raises(ValueError):
            md.md_combine_backward(dout, rows, w, y_rows=bad, dy=torch.empty_like(y))
    with pytest.raises(TypeError):
        md.md_combine_backward(dout, rows, w, y.tolist())
    with pytest.raises(ValueError):
        md.md_combine_backward(dout, rows, w, y[0].contiguous())
    dy, dw = md.md_combine_backward(dout, rows, w, y, y_rows=T * k)
    again = md.md_combine_backward(dout, rows, w, y)
    assert torch.equal(dy, again[0]) and torch.equal(dw, again[1])
