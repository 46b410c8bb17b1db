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
