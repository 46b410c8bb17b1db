"""The expert products' kernel forms, one by one and one behind another.

Which form a call takes goes by its shape, and the smaller shapes of the other expert tests all take the
few-row form; here those tests run again in the two forms for many rows, and in cases that
only these meet.  Tolerances are those of the other tests: 2^-8 |want| for the rounding to bf16 and
n 2^-23 S for a float32 sum of n products whose magnitudes add up to S; small integers are
held bit for bit."""
import numpy as np
import pytest
import torch

import combine_warp_top_router_b200 as md
import test_gpu_experts as base

from _util import DEV
from test_gpu_experts import close, groups, ints, owned, products64, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[md.MD_EXPERT_ONE, md.MD_EXPERT_TWO], ids=["one", "two"])
def pairs(request):
    """CTA pairs with one product to a tile, and with two."""
    md.md_set_expert_path(request.param)
    yield request.param
    md.md_set_expert_path(md.MD_EXPERT_AUTO)


@pytest.fixture(params=[md.MD_EXPERT_FEW, md.MD_EXPERT_ONE, md.MD_EXPERT_TWO], ids=["few", "one", "two"])
def form(request):
    md.md_set_expert_path(request.param)
    yield request.param
    md.md_set_expert_path(md.MD_EXPERT_AUTO)


def test_another_form_is_refused():
    for bad in (-1, 4):
        with pytest.raises(md.MoeDispatchError) as err:
            md.md_set_expert_path(bad)
        assert err.value.code == md.MD_ERR_ARG
    md.md_set_expert_path(md.MD_EXPERT_AUTO)


# ------------------------------------------------------------------ the other tests' cases

@pytest.mark.parametrize("layout", [md.MD_W_NK, md.MD_W_KN])
@pytest.mark.parametrize("counts,K,N", base.SHAPES)
def test_gemm(pairs, counts, K, N, layout):
    base.test_gemm(counts, K, N, layout)


@pytest.mark.parametrize("layout", [md.MD_W_NK, md.MD_W_KN])
@pytest.mark.parametrize("counts,K,N", [([7, 0, 33], 128, 136), ([260, 31, 0, 512], 320, 264), ([257, 300], 1032, 1048)])
def test_exact_on_small_integers_and_other_rows_left(pairs, counts, K, N, layout):
    base.test_gemm_is_exact_on_small_integers_and_leaves_other_rows(counts, K, N, layout)


@pytest.mark.parametrize("op", ["nk", "kn", "gated"])
@pytest.mark.parametrize("counts,K,N", [([500] + [0] * 62 + [3], 200, 136), ([1, 0, 2], 2056, 264), ([0, 64, 1, 0], 1000, 136),
                                        ([1] * 200 + [0] * 823 + [7], 72, 64), ([300] * 80, 64, 1032),
                                        ([257] * 9 + [0, 513], 456, 776)])
def test_exact_on_small_integers(form, counts, K, N, op):
    base.test_forms_are_exact_on_small_integers(counts, K, N, op)


def test_nan_and_inf_stay_in_their_row_and_expert(pairs):
    base.test_gemm_keeps_nan_and_inf_to_their_row_and_expert()


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("counts,K,F", base.GATED + [([300, 0, 700, 5], 648, 520)])
def test_gated(pairs, counts, K, F, keep):
    base.test_gated(counts, K, F, keep)


@pytest.mark.parametrize("counts,F", [([5, 0, 2], 40), ([300, 20], 96), ([33, 290], 392)])
def test_checkpoint_is_exact_where_the_sums_are(form, counts, F):
    base.test_checkpoint_is_exact_where_the_sums_are(counts, F)


def test_checkpoint_stores_inf_and_nan_as_nan(pairs):
    base.test_checkpoint_stores_inf_and_nan_as_nan()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 8, 8), ([0, 3, 0, 1], 136, 72), ([16, 17, 15, 0, 64, 65], 264, 264), ([300, 0, 257, 256, 1, 255], 392, 520),
    ([2, 1, 700], 1416, 200), ([63, 64, 65, 127, 129], 776, 1032)])
def test_wgrad(pairs, counts, N, K, dtype):
    base.test_wgrad(counts, N, K, dtype)


def test_bad_ranges_are_empty_and_reported(pairs):
    base.test_bad_ranges_are_empty_and_reported()


def test_rows_but_no_expert_has_any(pairs):
    base.test_rows_but_no_expert_has_any()


@pytest.mark.parametrize("op", ["nk", "kn", "gated", "wgrad"])
def test_many_tiles(pairs, op):
    base.test_many_tiles_of_two_products(op)


@pytest.mark.parametrize("hi", [1, 63, 130])
def test_wgrad_of_many_short_experts(pairs, hi):
    base.test_wgrad_of_many_short_experts(hi)


def test_a_layer_forward_and_backward(form):
    base.test_a_layer_forward_and_backward_against_autograd_in_64_bits()


def test_a_wait_that_runs_out(pairs):
    base.test_a_wait_that_runs_out_is_reported_and_leaves_the_gpu_usable()


# ------------------------------------------------------------------ long contractions and experts

@pytest.mark.parametrize("op", ["nk", "kn"])
def test_long_contractions_of_ragged_experts(form, op):
    """Rings that wrap many times, tiles of every remainder, the last weight tile part empty."""
    counts, K, N = [129, 0, 256, 31, 257, 1, 64, 770, 33], 2056, 1160
    off, cnt, rows, spans = groups(counts, seed=4, gap=2)
    nk = op == "nk"
    x, w = randn(1, rows, K), randn(2, *((len(counts), N, K) if nk else (len(counts), K, N)))
    st = md.new_status(DEV)
    y = md.md_expert_gemm(x, w, off, cnt, md.MD_W_NK if nk else md.MD_W_KN, dev_status=st)
    md.check_status(st)
    want, mags = products64(x, w, spans, nk)
    close(y, want, mags, K, owned(rows, spans))


@pytest.mark.parametrize("counts,N,K", [([5000, 0, 1153, 1152, 100, 2305], 264, 520), ([2400] * 6 + [1, 0, 64], 776, 264),
                                        ([3000, 63, 4100], 520, 24)])
def test_wgrad_of_long_experts(pairs, counts, N, K):
    """Several parts to an expert, between experts of one part or none: fresh, added twice, in bf16, and
    with rows of nobody between that are not numbers."""
    off, cnt, rows, spans = groups(counts, seed=5, gap=3)
    dy, x = ints(1, rows, N, hi=2), ints(2, rows, K, hi=2)
    mine = owned(rows, spans)
    dy[~mine], x[~mine] = float("inf"), float("nan")
    want = torch.zeros(len(counts), N, K, dtype=torch.float64, device=DEV)
    for e, o, c in spans:
        want[e] = dy[o:o + c].double().t() @ x[o:o + c].double()
    st = md.new_status(DEV)
    dw = md.md_expert_wgrad(dy, x, off, cnt, dev_status=st)
    md.check_status(st)
    assert torch.equal(dw.double(), want)
    for more in (2, 3):
        md.md_expert_wgrad(dy, x, off, cnt, dw=dw, accumulate=True)
        assert torch.equal(dw.double(), more * want)
    assert torch.equal(md.md_expert_wgrad(dy, x, off, cnt, out_dtype=torch.bfloat16), want.to(torch.bfloat16))


def test_wgrad_of_a_long_expert_is_as_exact_as_of_a_short_one(pairs):
    """Normal data, errors in the 2-norm.  An expert of 1152 rows is one part: 72 products of 16 rows, each
    addition off by 2^-23 of the larger of the running sum, 4 sqrt(i) times a product's deviation, and
    of a product, taken as 4 times it: sum(4 sqrt(i) + 4) = 1930 against the result's sqrt(1152) = 34 is
    57 * 2^-23.  Of 40 parts the errors are independent, so that relative to the sum they are as one part's,
    and 39 float32 additions round to nearest, independently too: sqrt(40) * 2^-24 holds them.  10% for
    chance (137,000 outputs).  Summed whole, the error grows with the number of products: 40 times."""
    N, K, one = 264, 520, 1152
    errs = []
    for parts in (1, 40):
        rows = parts * one
        off, cnt, rows, _ = groups([rows])
        dy, x = randn(parts, rows, N), randn(parts + 1, rows, K)
        want = dy.double().t() @ x.double()
        errs.append(float((md.md_expert_wgrad(dy, x, off, cnt)[0].double() - want).norm() / want.norm()))
    assert errs[0] < 57 * 2.0 ** -23, errs
    assert errs[1] < 1.1 * (errs[0] ** 2 + 40 * 2.0 ** -48) ** 0.5, errs


# ------------------------------------------------------------------ one behind another, extremes

def test_pairs_one_behind_another():
    """Short calls of the CTA pairs' kernel back to back, each block of one behind a block of
    another on the same SM, with the few-row form between: nothing that a pair left unfinished
    may reach the shared memory of the next."""
    counts = np.random.default_rng(3).integers(65, 140, 80).tolist()
    off, cnt, rows, spans = groups(counts, seed=3)
    K, N = 72, 272
    x, dy = ints(1, rows, K, hi=1), ints(2, rows, N, hi=1)
    w = ints(3, len(counts), N, K, hi=1)
    zero, full = torch.zeros(1, dtype=torch.int32, device=DEV), torch.full((1,), 64, dtype=torch.int32, device=DEV)
    calls = [lambda: md.md_expert_gemm(x, w, off, cnt), lambda: md.md_expert_gemm(dy, w, off, cnt, md.MD_W_KN),
             lambda: md.md_expert_wgrad(dy, x, off, cnt), lambda: md.md_expert_gated(x, w, off, cnt),
             lambda: md.md_expert_gemm(x[:64], w[:1], zero, full)]
    want = [c() for c in calls]
    for e, o, c in spans:
        assert torch.equal(want[0][o:o + c].double(), x[o:o + c].double() @ w[e].double().t())
        assert torch.equal(want[2][e].double(), dy[o:o + c].double().t() @ x[o:o + c].double())
    order = np.random.default_rng(4).integers(0, len(calls), 1500).tolist()
    got = [(i, calls[i]()) for i in order]
    wrong = sum((y.view(torch.uint8) != want[i].view(torch.uint8)).any().long() for i, y in got)
    assert int(wrong) == 0


def test_as_many_rows_as_there_may_be():
    """One expert with 2^31 - 4097 rows: 69 GB of the smallest rows, zero but at both ends and around
    the middle."""
    rows = 2 ** 31 - 4097
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 69 GB")
    x = torch.zeros(rows, 8, dtype=torch.bfloat16, device=DEV)
    parts = [slice(0, 700), slice(2 ** 30 - 300, 2 ** 30 + 300), slice(rows - 700, rows)]
    for i, p in enumerate(parts):
        x[p] = ints(i, p.stop - p.start, 8)
    w = ints(7, 1, 8, 8)
    y = torch.full((rows, 8), 9.0, dtype=torch.bfloat16, device=DEV)
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    st = md.new_status(DEV)
    md.md_expert_gemm(x, w, t([0, rows]), t([rows]), out=y, dev_status=st)
    md.check_status(st)
    for p in parts:
        assert torch.equal(y[p], (x[p].double() @ w[0].double().t()).to(torch.bfloat16))
        y[p] = 0
    whole = y.view(-1).view(torch.int64)
    for at in range(0, whole.numel(), 1 << 30):
        assert not bool(whole[at:at + (1 << 30)].any())
    del x, y, whole
    torch.cuda.empty_cache()


@pytest.mark.parametrize("E,rows,N", [(8, 100, 64), (3, 70, 64), (64, 9000, 1416)])
@pytest.mark.parametrize("op", ["nk", "kn", "gated"])
def test_ranges_that_overlap_far_write_nothing(E, rows, N, op):
    """Every expert claims all rows: more tiles than the rows can make."""
    K = 512 if E == 3 else 72  # E == 3: a contraction that CTAs share
    x = ints(1, rows, K)
    w = ints(2, *((E, K, N) if op == "kn" else (E, 2 * N if op == "gated" else N, K)))
    cnt = torch.full((E,), rows, dtype=torch.int32, device=DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    st = md.new_status(DEV)
    y = torch.full((rows, N), 9.0, dtype=torch.bfloat16, device=DEV)
    if op == "gated":
        md.md_expert_gated(x, w, off, cnt, out=y, dev_status=st)
    else:
        md.md_expert_gemm(x, w, off, cnt, md.MD_W_KN if op == "kn" else md.MD_W_NK, out=y, dev_status=st)
    assert int(st.item()) == md.MD_ERR_DATA
    assert bool((y == 9.0).all())


@pytest.mark.parametrize("lo,hi", [(-86, -60), (-60, -46), (-44, -16), (-16, 16), (16, 100)])
def test_activation_rounds_as_the_exact_one_but_next_to_a_border(lo, hi):
    """g sigma(g) u in float32 and one rounding to bf16, at a million arguments that float32 sums give
    exactly.  2^x is good to 4 * 2^-24, its correction to 1 and the float32 ln 2 in it to 4 for g > -87
    (1.9e-9 a unit of x), which makes 9 where g < -44; above, the last is 2 at most and the sum
    1 + 2^x (1) and its reciprocal (2) follow, which makes 10.  With two products: 12 * 2^-24.  Where the
    exact value is further from the border between two bf16 values, the result must be the nearer one."""
    rows, F, K = 32, 8192, 64
    g = torch.Generator(device=DEV).manual_seed(100 + lo)
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    x[torch.arange(rows), 2 * torch.arange(rows)] = 1
    x[torch.arange(rows), 2 * torch.arange(rows) + 1] = 1
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    wrong = near = 0
    for _ in range(4):
        # two summands each, 16 bits together: every order of summing is exact
        low = torch.randint(-127, 128, (2 * F, K), generator=g, device=DEV).double()
        w = torch.empty(2 * F, K, dtype=torch.float64, device=DEV)
        w[:F] = (lo + (hi - lo) * torch.rand(F, K, generator=g, device=DEV)).to(torch.bfloat16).double()
        w[F:] = ((1 + torch.rand(F, K, generator=g, device=DEV)) * 2.0 ** 20).to(torch.bfloat16).double()
        w[:F, 1::2] = low[:F, 1::2] * 2.0 ** -9
        w[F:, 1::2] = low[F:, 1::2] * 2.0 ** 5
        if lo == -16:  # 8 bits around 0 reach further down than 2^-9
            w[:F, 0::2] = (w[:F, 0::2] * 16).round() / 16
        act = md.md_expert_gated(x, w.to(torch.bfloat16)[None].contiguous(), t([0, rows]), t([rows]))
        h = (w[:, 0::2] + w[:, 1::2]).t()
        want = h[:, :F] / (1 + torch.exp(-h[:, :F])) * h[:, F:]
        tol = 12 * 2.0 ** -24 * want.abs()
        low_end, high_end = (want - tol).to(torch.bfloat16), (want + tol).to(torch.bfloat16)
        sure = low_end == high_end
        near += int((~sure).sum())
        wrong += int((sure & (act != low_end)).sum())
    assert near < 4 * rows * F * 0.01  # the borders' share: 2 * 12 * 2^-24 of 2^-8
    assert wrong == 0, wrong
