"""The MoE block's router gradient on the CPU: against automatic differentiation
of the gates g = s / sum s, s = sigmoid(z), in float64, and for tokens whose
picked scores are tiny or zero (whose gates are then 1/k, a constant)."""
import pytest

torch = pytest.importorskip("torch")

from fp8_block_scaled_sigmoid_amd import train  # noqa: E402


def _case(z):
    """float32 scores and gates as the router writes them (torch's own float32
    sigmoid is 0 from -89 on)."""
    s = torch.sigmoid(z.double()).float()
    total = s.sum(1, keepdim=True)
    gates = torch.where(total > 0, s / total, torch.full_like(s, 1.0 / s.shape[1]))
    return s, gates


@pytest.mark.parametrize("shift", [0.0, 4.0, 15.0, -15.0, -60.0])
def test_router_gradient(shift):
    gen = torch.Generator().manual_seed(1)
    z = torch.randn(50, 6, generator=gen) + shift
    dgate = torch.randn(50, 6, generator=gen)
    s, gates = _case(z)
    got = train.router_gradient(dgate, gates, s)
    z64 = z.double().requires_grad_(True)
    s64 = torch.sigmoid(z64)
    want, = torch.autograd.grad(s64 / s64.sum(1, keepdim=True), z64, dgate.double())
    # eight float32 roundings, three of them of gates and of 1 - s (absolute there)
    g = gates.double()
    mag = g * (dgate.abs() + (dgate * gates).abs().sum(1, keepdim=True))
    assert torch.all((got - want).abs() <= 16 * 2.0 ** -24 * mag)


def test_router_gradient_of_scores_that_are_zero():
    z = torch.tensor([[-200.0, -300.0, -1e4], [1.0, -200.0, 0.5], [-88.0, -89.0, -90.0]])
    dgate = torch.tensor([[1.0, -2.0, 3.0]] * 3)
    s, gates = _case(z)
    assert torch.all(s[0] == 0) and torch.all(gates[0] == gates[0, 0])
    got = train.router_gradient(dgate, gates, s)
    assert torch.isfinite(got).all()
    assert torch.all(got[0] == 0)           # the gates of this token do not move
    assert got[1, 1] == 0 and got[1, 0] != 0 and torch.all(got[2] != 0)


def test_router_gradient_of_no_tokens():
    e = torch.empty(0, 4)
    assert train.router_gradient(e, e, e).shape == (0, 4)


@pytest.mark.gpu
def test_block_gradients_with_a_token_that_no_expert_scores():
    """Token 0's logits underflow the sigmoid: its gates are 1/k, and every other
    gradient is that of the same block with its gates held constant."""
    from fp8_block_scaled_sigmoid_amd.train import BlockWeights, MoEBlock
    T, H, I, N, k = 24, 128, 64, 16, 2
    gen = torch.Generator(device="cuda").manual_seed(9)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(*shape, device="cuda").normal_(0, std, generator=gen).to(dtype)

    bf = torch.bfloat16
    router = (normal(N, H, std=0.3) - 1.0).to(bf)
    w = BlockWeights(router, normal(N, std=0.05), normal(N + 1, 2 * I, H, std=0.15, dtype=bf),
                     normal(N + 1, H, I, std=0.2, dtype=bf), torch.ones(H, device="cuda"),
                     torch.ones(H, device="cuda"), normal(H))
    x, dr = normal(T, H), normal(T, H)
    x -= x.mean(1, keepdim=True)        # the others do not see the router's mean
    x[0] = 1.0
    block = MoEBlock(w, k)
    print("MoEBlock with a token of zero scores", flush=True)
    _, _, saved = block.forward(x)
    idx, gates, scores = saved[2].long(), saved[3], saved[4]
    assert torch.all(scores[0] == 0) and torch.all(gates[0] == 1.0 / k)
    dx, _ = block.backward(saved, dr)

    p = {n: getattr(w, n).double().cpu().requires_grad_(True) for n in w.trained}
    xd = x.double().cpu().requires_grad_(True)

    def rms(v, weight):
        return v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + block.eps) * weight

    def expert(e, v):
        g, u = (v @ p["w1"][e].t()).chunk(2, -1)
        return (g * torch.sigmoid(g) * u) @ p["w2"][e].t()

    h = rms(xd, p["w_pre"])
    picked = idx.cpu()
    s = torch.sigmoid(h[1:] @ p["w_router"].t()).gather(1, picked[1:])
    g = torch.cat([torch.full((1, k), 1.0 / k, dtype=torch.float64), s / s.sum(1, keepdim=True)])
    rows = expert(N, h)
    for j in range(k):
        rows = rows + g[:, j:j + 1] * torch.stack([expert(int(picked[t, j]), h[t]) for t in range(T)])
    r = xd + p["gate"] * rms(rows, p["w_post"])
    want = torch.autograd.grad((r * dr.double().cpu()).sum(), [xd] + [p[n] for n in w.trained])
    for name, ref in zip(("x",) + w.trained, want):
        val = (dx if name == "x" else block.grads[name]).double().cpu()
        err = float((val - ref).norm() / ref.norm())
        print(f"{name}: relative L2 error {err:.2e}")
        assert err <= 10 * 2.0 ** -8, name      # ten bf16 roundings between, as for any block
