"""Calls on a stream other than the current one: what they allocate comes from
that stream's memory, and their results are those of the current stream."""
import pytest
import torch

from tests.gpu_util import log, require_gpu
from tests.ops_util import offsets_of

pytestmark = pytest.mark.gpu


def operator_calls(M):
    """name -> call(stream) with outputs of 2 MB and more."""
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    T, N, K = 4096, 512, 512
    x, dy, w, off = r(T, K).bfloat16(), r(T, N).bfloat16(), r(2, N, K).bfloat16(), offsets_of([T - 5, 5]).cuda()
    logits, d_w = r(T, 256), r(T, 64)
    ids, _ = M.router_topk(logits, 64)
    q, wq = M.mx_quant(x), M.mx_quant(w)
    return {
        "router_topk": lambda s: M.router_topk(logits, 64, stream=s),
        "router_topk_grad": lambda s: M.router_topk_grad(logits, ids, d_w, stream=s),
        "grouped_gemm": lambda s: M.grouped_gemm(x, w, off, stream=s),
        "grouped_gemm_dgrad": lambda s: M.grouped_gemm_dgrad(dy, w, off, stream=s),
        "grouped_gemm_wgrad": lambda s: M.grouped_gemm_wgrad(dy, x, off, out_dtype=torch.float32, stream=s),
        "mx_quant": lambda s: M.mx_quant(x, stream=s),
        "mx_dequant": lambda s: M.mx_dequant(*q, stream=s),
        "mx_grouped_gemm": lambda s: M.mx_grouped_gemm(*q, *wq, off, stream=s),
    }


def tensors(out):
    return out if isinstance(out, tuple) else (out,)


def test_operators_do_not_reuse_the_current_streams_memory():
    require_gpu()
    import w4a16_int4_grouped_amd as M
    side = torch.cuda.Stream()
    for name, call in operator_calls(M).items():
        log(f"case stream memory {name}")
        want = tensors(call(None))
        torch.cuda.synchronize()
        free = [torch.empty_like(t) for t in want]            # blocks of the same sizes, given back to this stream
        places = {t.data_ptr() for t in free}
        del free
        got = tensors(call(side))
        side.synchronize()
        assert not places & {t.data_ptr() for t in got}, name
        for a, b in zip(got, want):
            assert torch.equal(a, b), name


def test_the_layer_does_not_reuse_the_current_streams_memory():
    """Its output, and the workspace that it gives back on return: calls queued on two streams, bit for bit the calls
    made one at a time."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    from tests.test_gpu_n_operators import tiny_handle
    E, H, I, T, topk = 16, 1024, 512, 2000, 4
    log("case stream memory of the layer")
    h = tiny_handle(E, H, I)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    routes = [M.router_topk(torch.randn(T, E, generator=g, device="cuda"), topk, renorm=True) for _ in range(2)]
    want = [h.indexed(x, *r) for r in routes]
    nbytes = h.workspace_bytes(T, topk, T)
    torch.cuda.synchronize()
    free = [torch.empty_like(want[0]), torch.empty(nbytes, dtype=torch.uint8, device="cuda")]
    places = {t.data_ptr() for t in free}
    del free
    side = torch.cuda.Stream()
    got = [(h.indexed(x, *routes[k % 2], stream=side), h.indexed(x, *routes[1 - k % 2])) for k in range(4)]
    torch.cuda.synchronize()
    assert not places & {o.data_ptr() for o, _ in got}
    for k, (a, b) in enumerate(got):
        assert torch.equal(a, want[k % 2]) and torch.equal(b, want[1 - k % 2]), k


def test_side_stream_inside_a_capture():
    """Outputs made for a side stream while a graph is captured belong to the graph: replays with eager calls of the
    same sizes between them give the eager results."""
    require_gpu()
    import w4a16_int4_grouped_amd as M
    log("case side stream in a capture")
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    a, w1, w2, off = r(300, 256), r(3, 512, 256), r(3, 256, 512), offsets_of([100, 0, 200]).cuda()

    def both(side):
        """Two products on the side stream, a third of the caller's beside them."""
        if side is not None:
            side.wait_stream(torch.cuda.current_stream())
        hid = M.grouped_gemm(a, w1, off, stream=side)
        y = M.grouped_gemm(hid, w2, off, stream=side)
        mine = M.grouped_gemm(a, w1, off, out_dtype=torch.float32)
        if side is not None:
            torch.cuda.current_stream().wait_stream(side)
        return y + 1, mine

    side = torch.cuda.Stream()
    both(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both(side)
    for k in range(4):
        a.copy_(a.roll(1, 0))
        want = both(None)
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        both(side if k % 2 else None)
        torch.cuda.synchronize()
        for x, y in zip(outs, want):
            assert torch.equal(x, y), k
