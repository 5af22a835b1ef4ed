"""The balance loss and its gradient with the most tokens (2^24) and the most sequences (2^23)
they take, and a training step of the block with the loss, captured and replayed."""
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a device"
    import fp8_block_scaled_sigmoid_amd as m
    m.lib()
    return m


def _plain(s, idx, bounds, alpha):
    """(loss, load, prob, counts) per sequence in float64 on the device."""
    T, N = s.shape
    share = s.double() / s.double().sum(1, keepdim=True)
    out = []
    for lo, hi in zip(bounds[:-1], bounds[1:]):
        n = hi - lo
        counts = torch.bincount(idx[lo:hi].flatten().long(), minlength=N)
        load, prob = counts.double() * N / (idx.shape[1] * n), share[lo:hi].sum(0) / n
        out.append((alpha * (load * prob).sum(), load, prob, counts))
    return [torch.stack(v) for v in zip(*out)]


def test_the_most_tokens(moe):
    """2^24 tokens in tiles of 1024 (128 shares a lane and eight waves in float32)."""
    T, N, k = 1 << 24, 6, 2
    gen = torch.Generator(device="cuda").manual_seed(1)
    s = torch.rand(T, N, device="cuda", generator=gen) * 0.98 + 0.01
    idx = s.topk(k, 1).indices.int()
    bounds = [0, 12_345_678, T]
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    log("moe_balance_loss of 2^24 tokens")
    loss, st = moe.moe_balance_loss(s, idx, off, alpha=0.25)
    want, load, prob, counts = _plain(s, idx, bounds, 0.25)
    assert torch.equal(st.counts.long(), counts) and st.tokens.tolist() == [12_345_678, T - 12_345_678]
    assert ((st.load.double() - load).abs() <= U * load).all()
    rel = U * (N / 64 + 8 + 2 + 128 + 8)
    assert ((st.prob.double() - prob).abs() <= (rel + U) * prob).all()
    assert ((loss.double() - want).abs() <= (rel + U) * want).all()
    log("moe_router_backward of 2^24 tokens")
    dz = moe.moe_router_backward(s, idx, load=st.load, tokens=st.tokens, seq_offsets=off, alpha=1e6,
                                 out_dtype=torch.float32)
    for q, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
        for at in (lo, hi - 1000):
            v = s[at:at + 1000].double()
            a, f = v / v.sum(1, keepdim=True), st.load[q].double()
            dot = (a * f).sum(1, keepdim=True)
            c = 1e6 / (hi - lo)
            ref, mag = c * a * (1 - v) * (f - dot), c * a * (f + dot)
            assert ((dz[at:at + 1000].double() - ref).abs() <= U * (2 * N / 64 + 40) * mag).all()
    assert not dz.isnan().any() and dz.abs().sum(1).count_nonzero() > T - 100


def test_the_most_sequences(moe):
    """2^23 sequences of two tokens each but for an empty one at either end and a longer one."""
    S, N, k = 1 << 23, 4, 1
    T = 2 * (S - 2) + 3
    sizes = torch.full((S,), 2, dtype=torch.int64, device="cuda")
    sizes[0] = sizes[-1] = 0
    sizes[S // 2] = 5
    off = torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).int()
    assert off[-1].item() == T <= 1 << 24
    gen = torch.Generator(device="cuda").manual_seed(2)
    s = torch.rand(T, N, device="cuda", generator=gen) * 0.98 + 0.01
    idx = s.topk(k, 1).indices.int()
    log("moe_balance_loss of 2^23 sequences")
    loss, st = moe.moe_balance_loss(s, idx, off, alpha=1.0)
    assert torch.equal(st.tokens.long(), sizes)
    of = torch.repeat_interleave(torch.arange(S, device="cuda"), sizes)
    counts = torch.zeros(S * N, dtype=torch.int64, device="cuda")
    counts.scatter_add_(0, of * N + idx[:, 0].long(), torch.ones_like(of))
    assert torch.equal(st.counts.long().view(-1), counts)
    share = s.double() / s.double().sum(1, keepdim=True)
    first = off[:-1].long()
    prob = torch.zeros(S, N, dtype=torch.float64, device="cuda")
    for i in range(5):
        has = sizes > i
        prob[has] += share[first[has] + i]
    n = sizes.clamp(min=1)[:, None]
    prob, load = prob / n, counts.view(S, N) * N / n.double()
    rel = U * (N / 64 + 8 + 2 + 5)
    assert ((st.prob.double() - prob).abs() <= (rel + U) * prob).all()
    assert ((st.load.double() - load).abs() <= U * load).all()
    want = (load * prob).sum(1)
    assert ((loss.double() - want).abs() <= (rel + U) * want).all()
    log("moe_router_backward of 2^23 sequences")
    dz = moe.moe_router_backward(s, idx, load=st.load, tokens=st.tokens, seq_offsets=off, alpha=1.0,
                                 out_dtype=torch.float32)
    f, v = st.load.double()[of], s.double()
    dot = (share * f).sum(1, keepdim=True)
    c = 1 / sizes[of].double()[:, None]
    ref, mag = c * share * (1 - v) * (f - dot), c * share * (f + dot)
    assert ((dz.double() - ref).abs() <= U * (2 * N / 64 + 40) * mag).all()


def test_block_step_captured_and_replayed():
    """Forward and backward pass of the block with the loss in one graph, replayed on new inputs
    with eager steps of another block of the same weights between."""
    from fp8_block_scaled_sigmoid_amd.train import MoEBlock
    from test_gpu_train_balance import _weights
    T, H, I, N, k = 200, 128, 64, 16, 3
    w, x, dr = _weights(T, H, I, N, 12)
    off = torch.tensor([0, 70, 70, 200], dtype=torch.int32, device="cuda")
    mask = torch.arange(T, device="cuda") % 9 != 8
    dloss = torch.tensor([1.0, 2.0, -3.0], device="cuda")
    blocks = [MoEBlock(w, k, balance_alpha=4.0) for _ in range(2)]

    def step(block):
        r, _, saved = block.forward(x, seq_offsets=off, token_mask=mask)
        dx, _ = block.backward(saved, dr, dbalance=dloss)
        return r, dx, block.balance_loss(saved)
    step(blocks[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(blocks[0])
    for i in range(4):
        gen = torch.Generator(device="cuda").manual_seed(i)
        for t in (x, dr, dloss):
            t.normal_(generator=gen)
        log(f"MoEBlock with a balance loss, replay {i}")
        graph.replay()
        want = step(blocks[1])
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for n in w.trained:
            assert torch.equal(blocks[0].grads[n], blocks[1].grads[n]), n
