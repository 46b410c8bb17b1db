"""Host-side refusals of the expert operators' C entry points: an error code, nothing enqueued.

No argument is touched before it is refused, so the pointers here are only numbers
(aligned or not), and no GPU is needed."""
import pytest

from combine_warp_top_router_b200 import binding

ARG, UNSUPPORTED, OK = binding.MD_ERR_ARG, binding.MD_ERR_UNSUPPORTED, binding.MD_OK
P, ODD = 0x10000, 0x10008  # 16-byte aligned, and not


def L():
    return binding.lib()


def gemm(x=P, rows=10, K=64, w=P, E=4, N=64, layout=0, off=P, cnt=P, y=P):
    return L().md_expert_gemm(x, rows, K, w, E, N, layout, off, cnt, y, None, None)


def gated(x=P, rows=10, K=64, w=P, E=4, F=64, off=P, cnt=P, act=P, codes=P, scales=P):
    return L().md_expert_gated(x, rows, K, w, E, F, off, cnt, act, codes, scales, None, None)


def wgrad(dy=P, x=P, rows=10, E=4, N=64, K=64, off=P, cnt=P, kind=0, acc=0, dw=P):
    return L().md_expert_wgrad(dy, x, rows, E, N, K, off, cnt, kind, acc, dw, None, None)


def backward(da=P, codes=P, scales=P, rows=10, F=64, dh=P, act=P):
    return L().md_expert_gated_backward(da, codes, scales, rows, F, dh, act, None)


def combine(dout=P, y=P, y_rows=10, rows=P, w=P, T=5, k=2, H=64, dy=P, dw=P):
    return L().md_combine_backward(dout, y, y_rows, rows, w, T, k, H, dy, dw, None, None)


BAD = [
    (gemm, [dict(rows=-1), dict(K=0), dict(K=60), dict(K=-8), dict(N=0), dict(N=12), dict(E=0), dict(layout=2),
            dict(layout=-1), dict(x=None), dict(w=None), dict(y=None), dict(off=None), dict(cnt=None), dict(x=ODD),
            dict(w=ODD), dict(y=ODD)]),
    (gated, [dict(rows=-1), dict(K=12), dict(F=4), dict(F=0), dict(E=0), dict(codes=None), dict(scales=None),
             dict(codes=ODD), dict(act=ODD), dict(act=None), dict(x=ODD), dict(w=ODD), dict(cnt=None)]),
    (wgrad, [dict(rows=-1), dict(N=12), dict(K=0), dict(E=0), dict(kind=2), dict(kind=-1), dict(kind=1, acc=1),
             dict(dw=None), dict(dw=ODD), dict(dy=None), dict(x=ODD), dict(off=None)]),
    (backward, [dict(rows=-1), dict(F=0), dict(F=12), dict(da=None), dict(codes=None), dict(scales=None), dict(dh=None),
                dict(da=ODD), dict(codes=ODD), dict(dh=ODD), dict(act=ODD)]),
    (combine, [dict(T=-1), dict(k=0), dict(k=33), dict(H=0), dict(H=12), dict(y_rows=-1), dict(dout=None),
               dict(rows=None), dict(w=None), dict(dy=None), dict(y=None), dict(dout=ODD), dict(dy=ODD), dict(y=ODD)]),
]


@pytest.mark.parametrize("call,args", [(c, a) for c, many in BAD for a in many])
def test_bad_arguments(call, args):
    assert call(**args) == ARG


@pytest.mark.parametrize("call,args", [
    (gemm, dict(E=1025)), (gemm, dict(N=(1 << 20) + 8)), (gemm, dict(K=(1 << 20) + 8)),
    (gemm, dict(N=1 << 20, K=1 << 18)), (gemm, dict(rows=(1 << 31) - 4096)), (gated, dict(F=(1 << 19) + 8)),
    (gated, dict(E=2000)), (wgrad, dict(N=1 << 19, K=1 << 19)), (wgrad, dict(rows=1 << 33))])
def test_sizes_outside_the_limits(call, args):
    assert call(**args) == UNSUPPORTED


def test_calls_without_rows_enqueue_nothing():
    before = L().md_launch_count()
    assert gemm(rows=0, x=None, y=None) == OK
    assert gated(rows=0, x=None, act=None) == OK
    assert wgrad(rows=0, dy=None, x=None, acc=1) == OK
    assert backward(rows=0, da=None, codes=None, scales=None, dh=None) == OK
    assert combine(T=0, dout=None, rows=None, w=None) == OK
    assert L().md_launch_count() == before


@pytest.mark.parametrize("call,args", [
    (gemm, dict(y=P)), (gemm, dict(x=P, w=16 * P, y=P + 10 * 64 * 2 - 16)), (gemm, dict(x=16 * P, w=P, y=P + 4 * 64 * 64 * 2 - 16)),
    (gemm, dict(x=P + 16, w=16 * P, y=P)),
    (gated, dict(x=P, w=16 * P, act=P, codes=None, scales=None)), (gated, dict(x=P, w=16 * P, act=32 * P, codes=P + 1264, scales=64 * P)),
    (gated, dict(x=P, w=16 * P, act=32 * P, codes=48 * P, scales=16 * P + 4 * 128 * 64 * 2 - 1)),
    (gated, dict(x=P, w=16 * P, act=32 * P, codes=32 * P + 1264, scales=64 * P)),
    (gated, dict(x=P, w=16 * P, act=32 * P, codes=48 * P, scales=48 * P + 10 * 128 - 1)),
    (wgrad, dict(dy=P, x=16 * P, dw=P)), (wgrad, dict(dy=P, x=16 * P, dw=16 * P - 4 * 64 * 64 * 4 + 16)),
    (backward, dict(da=P, codes=2 * P, scales=3 * P, dh=4 * P, act=P)), (backward, dict(da=P, codes=2 * P, scales=3 * P, dh=P + 1264, act=None)),
    (backward, dict(da=P, codes=2 * P, scales=3 * P, dh=4 * P, act=4 * P + 2 * 1280 - 16)),
    (backward, dict(da=P, codes=2 * P, scales=4 * P + 2 * 1280 - 1, dh=4 * P, act=None)),
    (combine, dict(dout=2 * P, y=P, dy=P)), (combine, dict(dout=P, y=None, dw=None, dy=P + 5 * 64 * 2 - 16))])
def test_outputs_on_top_of_inputs_or_each_other(call, args):
    assert call(**args) == ARG
