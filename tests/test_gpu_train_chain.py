"""Two MoE blocks in a chain, the boundary between them in one pass each way (the
first block forms the second one's norm, and takes back that norm's gradient) or
each block with its own norm: outputs and every gradient against float64
automatic differentiation on the CPU.

Bar: twice that of a single block, about ten bf16 roundings each, 20 * 2^-8 of
the result's norm."""
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BAR = 20 * 2.0 ** -8
T, H, I, N, k = 40, 128, 64, 16, 3
ALPHA, BETA = 0.9, 0.8


def _weights(gen):
    from fp8_block_scaled_sigmoid_amd.train import BlockWeights
    bf = torch.bfloat16

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(*shape, device="cuda").normal_(0, std, generator=gen).to(dtype)

    return BlockWeights(normal(N, H, std=0.3, dtype=bf), normal(N, std=0.05),
                        normal(N + 1, 2 * I, H, std=0.15, dtype=bf), normal(N + 1, H, I, std=0.2, dtype=bf),
                        1 + normal(H, std=0.1), 1 + normal(H, std=0.1), normal(H))


def _block(p, x, idx, eps):
    def rms(v, weight):
        return v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + eps) * weight

    def expert(e, v):
        g, u = (v @ p["w1"][e].t()).chunk(2, -1)
        return (g * torch.sigmoid(g) * u) @ p["w2"][e].t()

    h = rms(x, p["w_pre"])
    s = torch.sigmoid(h @ p["w_router"].t()).gather(1, idx)
    gates = s / s.sum(1, keepdim=True)
    rows = expert(N, h)
    for j in range(k):
        rows = rows + gates[:, j:j + 1] * torch.stack([expert(int(idx[t, j]), h[t]) for t in range(T)])
    return ALPHA * x + BETA * p["gate"] * rms(rows, p["w_post"])


@pytest.mark.parametrize("joined", [True, False])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_two_blocks(stream, joined):
    from fp8_block_scaled_sigmoid_amd.train import MoEBlock
    gen = torch.Generator(device="cuda").manual_seed(41)
    one, two = (MoEBlock(_weights(gen), k, alpha=ALPHA, beta=BETA) for _ in range(2))
    dt = torch.bfloat16 if stream == "bf16" else torch.float32
    x, dr = (torch.empty(T, H, device="cuda").normal_(generator=gen).to(dt) for _ in range(2))
    w_pre = two.w.w_pre
    log(f"two MoEBlocks, {stream} stream, joined {joined}")
    if joined:
        r1, h1, s1 = one.forward(x, next_w_pre=w_pre)
        r2, _, s2 = two.forward(r1, h=h1)
        dr1, none, dh1 = two.backward(s2, dr, through_norm=False)
        dx, dw = one.backward(s1, dr1, dh_next=dh1, next_w_pre=w_pre, dw_next=two.grads["w_pre"])
        assert none is None and dw is two.grads["w_pre"]
    else:
        r1, _, s1 = one.forward(x)
        r2, _, s2 = two.forward(r1)
        dr1, _ = two.backward(s2, dr)
        dx, _ = one.backward(s1, dr1)

    xd = x.double().cpu().requires_grad_(True)
    p = [{n: getattr(b.w, n).double().cpu().requires_grad_(True) for n in b.w.trained} for b in (one, two)]
    out = xd
    for q, saved, b in zip(p, (s1, s2), (one, two)):
        out = _block(q, out, saved[2].long().cpu(), b.eps)
    names = [(i, n) for i in (0, 1) for n in p[i]]
    want = torch.autograd.grad((out * dr.double().cpu()).sum(), [xd] + [p[i][n] for i, n in names])
    got = [r2, dx] + [(one, two)[i].grads[n] for i, n in names]
    for name, val, ref in zip(["r", "x"] + names, got, [out.detach(), *want]):
        err = float((val.double().cpu() - ref).norm() / ref.norm())
        print(f"{name}: relative L2 error {err:.2e}")
        assert err <= BAR, name
