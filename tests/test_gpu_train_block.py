"""The MoE block in bf16 end to end: output and every gradient against float64
automatic differentiation of the same block on the CPU, and the training
example.

Bar: each result passes through at most about ten bf16 roundings (h, a, the
activation, the expert rows, b, db, dact, da, drows, dh), each of relative size
up to 2^-8; their effects add at most linearly, 10 * 2^-8 = 4e-2 of the
result's norm."""
import os
import sys

import numpy as np
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAR = 10 * 2.0 ** -8


def _reference(w, x, idx, k, alpha, beta, eps, dr, next_w, dh_next):
    """Gradients by automatic differentiation in float64, for the given picks."""
    p = {n: getattr(w, n).double().cpu().requires_grad_(True) for n in w.trained}
    x = x.double().cpu().requires_grad_(True)
    nw = next_w.double().cpu().requires_grad_(True)

    def rms(v, weight):
        return v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + eps) * weight

    h = rms(x, p["w_pre"])
    s = torch.sigmoid(h @ p["w_router"].t()).gather(1, idx)
    gates = s / s.sum(1, keepdim=True)

    def expert(e, v):
        g, u = (v @ p["w1"][e].t()).chunk(2, -1)
        return (g * torch.sigmoid(g) * u) @ p["w2"][e].t()

    rows = [expert(w.N, h)]
    for j in range(k):
        out = torch.stack([expert(int(idx[t, j]), h[t]) for t in range(len(x))])
        rows.append(gates[:, j:j + 1] * out)
    r = alpha * x + beta * p["gate"] * rms(sum(rows), p["w_post"])
    hn = rms(r, nw)
    loss = (r * dr.double().cpu()).sum() + (hn * dh_next.double().cpu()).sum()
    names = list(p)
    got = torch.autograd.grad(loss, [x, nw] + [p[n] for n in names])
    return r.detach(), hn.detach(), dict(zip(["x", "next"] + names, got))


@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_block_gradients(stream):
    from fp8_block_scaled_sigmoid_amd.train import BlockWeights, MoEBlock
    T, H, I, N, k = 40, 128, 64, 16, 3
    gen = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(*shape, device="cuda").normal_(0, std, generator=gen).to(dtype)

    bf = torch.bfloat16
    w = BlockWeights(normal(N, H, std=0.3, dtype=bf), normal(N, std=0.05),
                     normal(N + 1, 2 * I, H, std=0.15, dtype=bf), normal(N + 1, H, I, std=0.2, dtype=bf),
                     1 + normal(H, std=0.1), 1 + normal(H, std=0.1), normal(H))
    dt = bf if stream == "bf16" else torch.float32
    x, dr = normal(T, H, dtype=dt), normal(T, H, dtype=dt)
    dh_next, next_w = normal(T, H, dtype=bf), 1 + normal(H, std=0.1)
    block = MoEBlock(w, k, alpha=0.9, beta=0.8)
    log(f"MoEBlock forward and backward, {stream} stream")
    r, h_next, saved = block.forward(x, next_w_pre=next_w)
    dx, dw_next = block.backward(saved, dr, dh_next, next_w)
    rr, hr, want = _reference(w, x, saved[2].long().cpu(), k, 0.9, 0.8, block.eps, dr, next_w, dh_next)
    got = {"x": dx, "next": dw_next, **block.grads}
    for name, ref in {"r": rr, "h_next": hr, **want}.items():
        val = {"r": r, "h_next": h_next}.get(name, got.get(name)).double().cpu()
        err = float((val - ref).norm() / ref.norm())
        print(f"{name}: relative L2 error {err:.2e}")
        assert err <= BAR, name
    total = float(torch.cat([t.double().reshape(-1) for t in block.grads.values()]).norm())
    result = block.clip(0.1).cpu().numpy()
    assert abs(result[0] - total) <= 1e-5 * total
    after = float(torch.cat([t.double().reshape(-1) for t in block.grads.values()]).norm())
    assert abs(after - 0.1) <= 1e-5


def test_block_one_token():
    """One token: nearly every expert has no rows, and its gradient is zero."""
    from fp8_block_scaled_sigmoid_amd.train import BlockWeights, MoEBlock
    H, I, N, k = 256, 64, 32, 2
    gen = torch.Generator(device="cuda").manual_seed(6)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(*shape, device="cuda").normal_(0, std, generator=gen).to(dtype)

    bf = torch.bfloat16
    w = BlockWeights(normal(N, H, std=0.3, dtype=bf), normal(N, std=0.05),
                     normal(N + 1, 2 * I, H, std=0.15, dtype=bf), normal(N + 1, H, I, std=0.2, dtype=bf),
                     1 + normal(H, std=0.1), 1 + normal(H, std=0.1), normal(H))
    x, dr, dh_next = normal(1, H), normal(1, H), normal(1, H, dtype=bf)
    next_w = 1 + normal(H, std=0.1)
    block = MoEBlock(w, k)
    log("MoEBlock forward and backward, one token")
    r, h_next, saved = block.forward(x, next_w_pre=next_w)
    dx, dw_next = block.backward(saved, dr, dh_next, next_w)
    idx = saved[2].long().cpu()
    rr, hr, want = _reference(w, x, idx, k, 1.0, 1.0, block.eps, dr, next_w, dh_next)
    got = {"r": r, "h_next": h_next, "x": dx, "next": dw_next, **block.grads}
    for name, ref in {"r": rr, "h_next": hr, **want}.items():
        err = float((got[name].double().cpu() - ref).norm() / ref.norm())
        print(f"{name}: relative L2 error {err:.2e}")
        assert err <= BAR, name
    unused = [e for e in range(N) if e not in idx[0].tolist()]
    assert torch.all(block.grads["w1"][unused] == 0) and torch.all(block.grads["w2"][unused] == 0)


def test_training_example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_block
    finally:
        sys.path.pop(0)
    log("examples/train_block.py")
    losses = train_block.train(tokens=256, steps=12)
    assert np.all(np.isfinite(losses)) and losses[-1] < 0.9 * losses[0]
