"""Calls on a stream of their own (stream=) that allocate their scratch and
results themselves: the current stream allocates and writes meanwhile, and the
results are the bits of a call on the current stream."""
import numpy as np
import pytest

from helpers import log, to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a device"
    import fp8_block_scaled_sigmoid_amd as m
    m.lib()
    return m


def _normal(gen, *shape, dtype=torch.bfloat16):
    return torch.empty(*shape, device="cuda", dtype=dtype).normal_(generator=gen)


def _offsets(sizes):
    return to_dev(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32))


def _product(moe, gen):
    sizes = [700, 1, 0, 2000, 33, 900]          # 15 row tiles x 24: counters in the scratch
    R, n, k = sum(sizes), 6144, 136
    assert moe.moe_grouped_gemm_bf16_workspace_bytes(len(sizes), R, n, k) > 0
    a, b, off = _normal(gen, R, k), _normal(gen, len(sizes), n, k), _offsets(sizes)
    return lambda **kw: [moe.moe_grouped_gemm_bf16(a, b, off, R, **kw)]


def _weight_gradient(moe, gen):
    R, n, k = 5000, 64, 136                     # cut into parts: partial sums in the scratch
    assert moe.moe_grouped_wgrad_bf16_workspace_bytes(1, R, n, k) > 0
    a, b, off = _normal(gen, R, n), _normal(gen, R, k), _offsets([R])
    return lambda **kw: [moe.moe_grouped_wgrad_bf16(a, b, off, R, **kw)]


def _norm_backward(moe, gen):
    r, dr, dh, b = (_normal(gen, 3000, 1032) for _ in range(4))
    w, gate = _normal(gen, 1032, dtype=torch.float32), _normal(gen, 1032, dtype=torch.float32)
    return lambda **kw: moe.moe_block_norm_backward(r, dr, dh, b, w, w, gate, **kw)


def _permutation(moe, gen):
    idx = torch.rand(4096, 64, device="cuda", generator=gen).topk(8, 1).indices.int()
    return lambda **kw: moe.moe_permute(idx, 64, **kw)


@pytest.mark.parametrize("make", [_product, _weight_gradient, _norm_backward, _permutation])
def test_scratch_of_a_call_on_another_stream(moe, make):
    gen = torch.Generator(device="cuda").manual_seed(21)
    call = make(moe, gen)
    want = [t.clone() for t in call()]
    busy = _normal(gen, 4096, 4096)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    log(f"{make.__name__} on another stream, its scratch allocated by the call")
    with torch.cuda.stream(s):
        for _ in range(20):                     # the call waits behind these
            busy @ busy
    got = call(stream=s)
    held = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
            for n in (512, 4096, 1 << 20, 4 << 20, 16 << 20) for _ in range(6)]
    torch.cuda.current_stream().wait_stream(s)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert all(bool((h == 255).all()) for h in held)


def test_list_dropped_behind_a_call_on_another_stream(moe):
    gen = torch.Generator(device="cuda").manual_seed(22)
    grads = [_normal(gen, n, dtype=torch.float32) for n in (5, 4096, 100001, 1, 30000)]
    outs = [torch.empty_like(g) for g in grads]
    want = moe.moe_grad_clip(moe.GradList(grads, outs), 0.5).clone()
    kept = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    busy = _normal(gen, 4096, 4096)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    log("moe_grad_clip of a list that is dropped, on another stream")
    with torch.cuda.stream(s):
        for _ in range(20):
            busy @ busy
    got = moe.moe_grad_clip(moe.GradList(grads, outs), 0.5, stream=s)
    held = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (200, 512) for _ in range(8)]
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want) and all(torch.equal(o, k) for o, k in zip(outs, kept))
    assert all(bool((h == 255).all()) for h in held)


def test_replays_of_a_captured_step(moe):
    """A graph of the operators, replayed with other inputs and eager work in
    between: the bits of the eager calls on every replay."""
    gen = torch.Generator(device="cuda").manual_seed(23)
    sizes, n, k = [700, 1, 0, 2000, 33, 900], 6144, 136      # the products take tiles from counters
    R, G, off = sum(sizes), len(sizes), _offsets(sizes)
    w = _normal(gen, G, n, k)
    x, x0, dy = _normal(gen, R, k), _normal(gen, R, k), _normal(gen, R, n)
    gain = _normal(gen, k, dtype=torch.float32)
    one = _offsets([R])
    dw = torch.empty(G, n, k, device="cuda")
    grads = moe.GradList([dw[e] for e in range(G)])

    def step():
        r, h = moe.moe_block_norm(x0, x, gain, gain, gain)
        a = moe.moe_grouped_gemm_bf16(h, w, off, R)
        act = moe.moe_swiglu(a)
        da, dgate, hg = moe.moe_swiglu_backward(a, dy[:, :n // 2])
        dh = moe.moe_grouped_gemm_bf16(da, w, off, R, b_kn=True)
        moe.moe_grouped_wgrad_bf16(da, h, off, R, out=dw)
        parts = moe.moe_grouped_wgrad_bf16(h, x, one, R)     # cut into parts
        back = moe.moe_block_norm_backward(r, x0, dh, x, gain, gain, gain)
        result = moe.moe_grad_clip(grads, 0.5)
        return [r, h, a, act, da, dgate, hg, dh, parts, *back, result, dw]

    assert moe.moe_grouped_gemm_bf16_workspace_bytes(G, R, n, k) > 0
    assert moe.moe_grouped_wgrad_bf16_workspace_bytes(1, R, k, k) > 0
    log("a captured step of the training operators")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(4):
        x.normal_(generator=gen)
        x0.normal_(generator=gen)
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        for t, u in zip(got, step()):
            assert torch.equal(t, u)
