"""A call on another stream than the current one: it must not write into memory that the current stream's
kernels still use, and its results are those of the current stream's call."""
import pytest
import torch

import combine_warp_top_router_b200 as md

from _util import DEV

pytestmark = pytest.mark.gpu

ROWS, N, E = 8192, 1024, 4  # outputs of 16 MB and more


def _calls():
    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    cnt = torch.full((E,), ROWS // E, dtype=torch.int32, device=DEV)
    off = torch.arange(E + 1, dtype=torch.int32, device=DEV) * (ROWS // E)
    x, w, dy = r(ROWS, 64), r(E, N, 64), r(ROWS, N)
    wide, codes_of = r(E, 2 * N, 64), md.md_expert_gated(x, r(E, 2 * N, 64), off, cnt, keep=True)[1:]
    rows = torch.arange(ROWS, dtype=torch.int32, device=DEV).view(-1, 2)
    idx = (rows % E).to(torch.int32)
    gates = torch.rand(ROWS // 2, 2, generator=g, device=DEV)
    logits = torch.randn(1 << 17, 64, generator=g, device=DEV)
    return {
        "gemm": (lambda s: md.md_expert_gemm(x, w, off, cnt, stream=s), ROWS * N * 2),
        "gated": (lambda s: md.md_expert_gated(x, wide, off, cnt, stream=s), ROWS * N * 2),
        "wgrad": (lambda s: md.md_expert_wgrad(dy, dy, off, cnt, stream=s), E * N * N * 4),
        "gated backward": (lambda s: md.md_expert_gated_backward(dy, *codes_of, want_act=False, stream=s)[0], ROWS * N * 4),
        "combine backward": (lambda s: md.md_combine_backward(dy[:ROWS // 2], rows, gates, stream=s)[0], ROWS * N * 2),
        "permute": (lambda s: md.md_dispatch_permute(dy[:ROWS // 2], rows, out_rows=ROWS, stream=s), ROWS * N * 2),
        "combine": (lambda s: md.md_combine(dy, rows, idx, gates, stream=s), ROWS // 2 * N * 2),
        "gather": (lambda s: md.md_gather_rows(dy, rows.view(-1), stream=s), ROWS * N * 2),
        "topk": (lambda s: md.md_route_topk(logits, 8, stream=s)[0], (1 << 17) * 8 * 4),
    }


@pytest.mark.parametrize("name", ["gemm", "gated", "wgrad", "gated backward", "combine backward", "permute", "combine",
                                  "gather", "topk"])
def test_memory_that_the_current_stream_still_reads(name):
    call, size = _calls()[name]
    side = torch.cuda.Stream()
    want = call(None)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = torch.full((size,), 5, dtype=torch.uint8, device=DEV)
    kept = torch.empty_like(freed)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    kept.copy_(freed)               # reads it when the call on the other stream has long run
    del freed
    got = call(side)
    torch.cuda.synchronize()
    assert bool((kept == 5).all())
    assert torch.equal(got, want)
