"""The balance loss and its gradient at sizes where the loss runs in tiles of many tokens and
where a lane has up to 16 experts, against the float64 oracle.

A tile of t tokens is max(16, min(1024, T / 256)) tokens.  Bars, in units of 2^-24 of values
whose terms are all positive: a token's share is a sum of N scores (N / 64 additions in a
lane, eight over the wave), a reciprocal and a product; a wave adds ceil(t / 8) shares in
float32, then eight waves are added; from there on sums are in double, and the result is
rounded once.  counts, tokens exact; load rounded once.  dz: as in
``test_gpu_router_balance``."""
import numpy as np
import pytest

from helpers import log, to_dev
from oracle import balance

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
KINDS = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a device"
    import fp8_block_scaled_sigmoid_amd as m
    m.lib()
    return m


CASES = [
    # T, N, k, sequence offsets (None: one of all tokens), masked
    (16384, 256, 8, None, False),
    (16384, 256, 8, [0, 5000, 5001, 5001, 9000, 12345, 16384], True),
    (20001, 64, 6, [0, 79, 80, 20001], True),                # tiles of 79 tokens and a rest
    (9000, 300, 4, [100, 4000, 8950], False),                # tokens of no sequence
    (300001, 16, 2, [0, 1024, 1025, 150000, 300001], False),         # tiles of 1024
    (200, 600, 8, [0, 63, 64, 130, 200], True),
    (700, 1024, 32, [0, 300, 300, 700], False),
    (333, 513, 3, None, True),
]


def _inputs(case):
    T, N, k, off, masked = case
    rng = np.random.default_rng(T * 5 + N + k)
    s = (1 / (1 + np.exp(-rng.standard_normal((T, N)) * 2))).astype(np.float32)
    s[7] = 0.0                                              # no expert scores this token
    idx = np.argpartition(-s, k - 1, 1)[:, :k].astype(np.int32)
    s[9, idx[9]] = 0.0                                      # nor its picks this one
    mask = (rng.random(T) < 0.7).astype(np.uint8) if masked else None
    if masked and off and len(off) > 3:
        mask[off[1]:off[2]] = 0                             # a sequence of padding alone
    dev = {"scores": to_dev(s), "idx": to_dev(idx),
           "seq_offsets": None if off is None else to_dev(np.array(off, np.int32)),
           "token_mask": None if mask is None else to_dev(mask)}
    return rng, s, idx, mask, dev


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[:3]}")
def test_loss(moe, case):
    T, N, k, off, masked = case
    _, s, idx, mask, dev = _inputs(case)
    log(f"moe_balance_loss in tiles {case}")
    loss, st = moe.moe_balance_loss(**dev, alpha=0.01)
    want = balance.router_balance(s, idx, off, mask, float(np.float32(0.01)))
    assert np.array_equal(st.counts.cpu().numpy(), want[3])
    assert np.array_equal(st.tokens.cpu().numpy(), want[4])
    assert np.all(np.abs(st.load.double().cpu().numpy() - want[1]) <= U * want[1])
    tile = max(16, min(1024, -(-T // 256)))
    rel = U * (N / 64 + 8 + 2 + -(-tile // 8) + 8)
    assert np.all(np.abs(st.prob.double().cpu().numpy() - want[2]) <= (rel + U) * want[2])
    assert np.all(np.abs(loss.double().cpu().numpy() - want[0]) <= (rel + U) * want[0])


@pytest.mark.parametrize("case", [c for c in CASES if c[0] < 10000], ids=lambda c: f"{c[:3]}")
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_gradient(moe, case, kind):
    T, N, k, off, masked = case
    rng, s, idx, mask, dev = _inputs(case)
    picked = np.take_along_axis(s, idx, 1)
    total = picked.sum(1, keepdims=True)
    gate = np.where(total > 0, picked / np.where(total > 0, total, 1), 1 / k).astype(np.float32)
    _, load, _, _, tokens = balance.router_balance(s, idx, off, mask)
    load = load.astype(np.float32)
    dgate = rng.standard_normal((T, k)).astype(np.float32)
    dloss = rng.standard_normal(len(tokens)).astype(np.float32)
    log(f"moe_router_backward {case} {kind}")
    dz = moe.moe_router_backward(**dev, gate=to_dev(gate), dgate=to_dev(dgate), load=to_dev(load),
                                 tokens=to_dev(tokens.astype(np.int32)), dloss=to_dev(dloss), alpha=3.0,
                                 out_dtype=KINDS[kind])
    want, mag = balance.router_backward(s, idx, gate.astype(np.float64), dgate.astype(np.float64),
                                        load.astype(np.float64), tokens, off, mask, dloss.astype(np.float64), 3.0)
    bar = HALF[kind] * np.abs(want) + U * (2 * N / 64 + 40) * mag
    assert np.all(np.abs(dz.double().cpu().numpy() - want) <= bar + 1e-42)


def test_two_graphs_share_a_workspace(moe):
    """Two captured losses on one workspace, replayed in turn with eager calls on it between."""
    T, N, k = 9000, 96, 4
    gen = torch.Generator(device="cuda").manual_seed(8)
    scores = torch.rand(T, N, device="cuda", generator=gen)
    idx = scores.topk(k, 1).indices.int()
    offs = [to_dev(np.array(o, np.int32)) for o in ([0, 4000, 9000], [0, 100, 7000])]
    need = moe.moe_balance_loss_workspace_bytes(T, N, 2)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    run = lambda o, **kw: moe.moe_balance_loss(scores, idx, o, **kw)        # noqa: E731
    run(offs[0], ws=ws)
    torch.cuda.synchronize()
    graphs = []
    for o in offs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            loss, st = run(o, ws=ws)
        graphs.append((g, o, loss, st))
    for step in range(4):
        scores.copy_(torch.rand(T, N, device="cuda", generator=gen))
        idx.copy_(scores.topk(k, 1).indices)
        log(f"balance losses that share a workspace, replay {step}")
        for g, o, loss, st in graphs:
            g.replay()
            eager, est = run(o, ws=ws)
            want, wst = run(o)
            torch.cuda.synchronize()
            assert torch.equal(loss, want) and torch.equal(eager, want)
            assert torch.equal(st.prob, wst.prob) and torch.equal(st.counts, wst.counts)
