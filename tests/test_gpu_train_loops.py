"""The training operators at sizes where every loop of their kernels makes more
than one round: tiles from the counters, rows behind a workgroup's first,
several chunks and tensors a workgroup.  Bars as in test_gpu_train."""
import numpy as np
import pytest

from helpers import log, to_dev
from oracle import train
from test_gpu_train import EPS, FLT, UB, _close, _make, _norm_inputs, _offsets, moe  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# ---------------------------------------------------------------------------
# grouped products whose workgroups take several tiles from the XCDs' counters

LISTS = {
    # 42 row tiles of nine column tiles
    "uneven": ([9000, 0, 5, 1200, 300, 0, 257, 31, 0], 2056),
    "one group": ([12000], 2056),
    "even": ([400] * 33, 1288),
    # the bound is 83 row tiles: 70 of one unit and a half each
    "small groups": ([49] * 70, 1032),
    # 13 row tiles at most of the 83: most workgroups find every list taken
    "all in one": ([0] * 40 + [3500] + [0] * 29, 1032),
    "two ends": ([1800] + [0] * 60 + [1700], 1288),
    # 70 groups of 257 and 1 rows: row tiles of 288 rows beside tiles of one
    "rests": ([257, 1] * 35, 776),
}


@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("name", list(LISTS))
def test_grouped_gemm_bf16_takes_tiles_from_the_counters(moe, name, kn):  # noqa: F811
    sizes, n = LISTS[name]
    off, k = _offsets(sizes), 72
    R, G = int(off[-1]), len(sizes)
    assert moe.moe_grouped_gemm_bf16_workspace_bytes(G, R, n, k) > 0
    rng = np.random.default_rng(R + n)
    gather = kn == (name in ("uneven", "small groups", "rests"))
    src = 501 if gather else R
    a, b = _make(rng, (src, k), "bf16"), _make(rng, (G, k, n) if kn else (G, n, k), "bf16", 0.1)
    index = rng.integers(0, src, R).astype(np.int32) if gather else None
    s = rng.standard_normal(R).astype(np.float32)
    out = "f32" if kn else "bf16"
    odt = torch.float32 if kn else torch.bfloat16
    log(f"moe_grouped_gemm_bf16 tiles from the counters, {name}, kn {kn}")
    args = (a[0], b[0], to_dev(off), R)
    kw = dict(b_kn=kn, a_row_index=to_dev(index) if gather else None, row_scale=to_dev(s))
    o = torch.full((R, n), float("nan"), dtype=odt, device="cuda")
    moe.moe_grouped_gemm_bf16(*args, out=o, **kw)
    want, mag = train.grouped_gemm(a[1], b[1], off, index, s, kn)
    _close(o, want, UB[out] * np.abs(want) + (k + 8) * 2.0 ** -23 * mag, "out")
    ws = torch.empty(moe.moe_grouped_gemm_bf16_workspace_bytes(G, R, n, k), dtype=torch.uint8,
                     device="cuda")
    for _ in range(3):              # which workgroup takes which tile changes nothing
        assert torch.equal(moe.moe_grouped_gemm_bf16(*args, out_dtype=odt, ws=ws, **kw), o)


# ---------------------------------------------------------------------------
# norms

ROUNDS = [
    # T, H, x, b, gate, post norm, pre norm: rows beyond those of 256 workgroups
    (600, 7168, "bf16", "bf16", "channel", True, True),
    (1021, 7168, "bf16", "bf16", "token", True, True),
    (515, 7168, "f32", "bf16", "full", True, True),
    (1021, 2049, "f32", "bf16", "full", True, True),
    (1700, 2049, "bf16", "f32", "channel", True, True),
    (513, 16384, "f32", "f32", "channel", True, True),
    (600, 8200, "bf16", "bf16", "full", True, True),
    (9001, 64, "bf16", "bf16", "channel", True, True),
    (5000, 513, "f32", "f32", "token", True, True),
    (2100, 1032, "bf16", "bf16", "none", False, True),
    (2100, 1032, "bf16", "bf16", "token", True, False),
]


@pytest.mark.parametrize("case", ROUNDS, ids=str)
def test_block_norm_backward_goes_round_its_rows(moe, case):  # noqa: F811
    T, H, xk, bk, gate, post, pre = case
    rng = np.random.default_rng(T * 41 + H)
    r, b, wq, wp, g = _norm_inputs(rng, T, H, xk, bk, gate, post, pre)
    dr = _make(rng, (T, H), xk, 0.1)
    dh = _make(rng, (T, H), bk, 0.1) if pre else (None, None)
    log(f"moe_block_norm_backward more rows than workgroups hold {case}")
    args = (r[0], dr[0], dh[0], b[0], wq[0], wp[0], g[0])
    got = moe.moe_block_norm_backward(*args, alpha=0.8, beta=0.6, eps=EPS)
    want = train.block_norm_backward(r[1], dr[1], dh[1], b[1], wq[1], wp[1], g[1],
                                     np.float32(0.8), np.float32(0.6), EPS)
    kinds = {"dx": xk, "db": bk, "dw_pre": "f32", "dw_post": "f32",
             "dgate": bk if gate == "full" else "f32"}
    for name, t in zip(("dx", "db", "dw_pre", "dw_post", "dgate"), got):
        if name not in want:
            assert t is None, name
            continue
        chain = FLT + (T + H if name.startswith("dw") or name == "dgate" else 0) * 2.0 ** -24
        _close(t, want[name], UB[kinds[name]] * np.abs(want[name]) + chain * want["mag"][name], name)
    again = moe.moe_block_norm_backward(*args, alpha=0.8, beta=0.6, eps=EPS)
    for t, u in zip(got, again):
        assert t is None or torch.equal(t, u)


def test_block_norm_backward_in_place_goes_round_its_rows(moe):  # noqa: F811
    T, H = 1021, 7168
    gen = torch.Generator(device="cuda").manual_seed(31)
    r, dr, dh, b = (torch.empty(T, H, device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
                    for _ in range(4))
    w, gate = (torch.empty(H, device="cuda").normal_(generator=gen) for _ in range(2))
    log("moe_block_norm_backward in place, four rounds of rows")
    want = moe.moe_block_norm_backward(r, dr, dh, b, w, w, gate)
    got = moe.moe_block_norm_backward(r, dr, dh, b, w, w, gate, dx=dr, db=b)
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("gate", ["token", "full"])
def test_block_norm_with_a_block_output_goes_round_its_rows(moe, gate):  # noqa: F811
    H, T = 8, (8 << 20) + 13
    gen = torch.Generator(device="cuda").manual_seed(32)
    x, b = (torch.empty(T, H, device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
            for _ in range(2))
    w = torch.empty(H, device="cuda").normal_(generator=gen)
    g = torch.empty(T, 1, device="cuda") if gate == "token" else torch.empty_like(b)
    g.normal_(generator=gen)
    log(f"moe_block_norm {T} x {H} with a block output and a gate per {gate}")
    r, h = moe.moe_block_norm(x, b, w, w, g, alpha=0.7, beta=0.4)
    for rows in (slice(0, 9), slice(T - 300, T)):
        r1, h1 = moe.moe_block_norm(x[rows], b[rows], w, w, g[rows], alpha=0.7, beta=0.4)
        assert torch.equal(r[rows], r1) and torch.equal(h[rows], h1)


# ---------------------------------------------------------------------------
# clipping: more than 2048 chunks of 4096 elements


def _long_list(gen, mixed):
    sizes = [3, 20_000_003, 1, 0, 4096, 4097] + [1 + 97 * i % 6000 for i in range(900)] + [5_000_001, 2]
    kinds = [torch.bfloat16 if mixed and i % 2 else torch.float32 for i in range(len(sizes))]
    flat = {d: torch.empty(sum(s for s, e in zip(sizes, kinds) if e is d) + 8, device="cuda",
                           dtype=d).normal_(0.0, 0.1, generator=gen)
            for d in set(kinds)}
    at, grads = {d: 1 for d in flat}, []        # one behind the other, at odd addresses
    for s, d in zip(sizes, kinds):
        grads.append(flat[d][at[d]:at[d] + s])
        at[d] += s
    return grads


@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("in_place", [True, False])
def test_grad_clip_of_a_long_list(moe, mixed, in_place):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(33)
    grads = _long_list(gen, mixed)
    before = [t.clone() for t in grads]
    values = [t.double().cpu().numpy() for t in grads]
    outs = None if in_place else [torch.full_like(t, 7.0) for t in grads]
    lst = moe.GradList(grads, outs)
    assert lst.chunks > 3 * 2048
    log(f"moe_grad_clip of {lst.chunks} chunks, mixed {mixed}, in place {in_place}")
    norm, coef = train.clip(values, 5.0)
    sumsq, n32 = moe.moe_grad_norm(lst)
    # squares of 24-bit values are exact in double; 1e-12 covers the sum's order
    assert abs(float(sumsq[0]) - norm ** 2) <= 1e-12 * norm ** 2
    assert abs(float(n32[0]) - norm) <= 2.0 ** -24 * norm + 1e-12 * norm
    result = moe.moe_grad_clip(lst, 5.0).cpu().numpy().astype(np.float64)
    assert abs(result[0] - norm) <= 2.0 ** -23 * norm
    assert abs(result[1] - coef) <= 2.0 ** -21 * coef
    for i, (t, v, o) in enumerate(zip(before, values, grads if in_place else outs)):
        if not in_place:
            assert torch.equal(grads[i], t)
        kind = "bf16" if o.dtype == torch.bfloat16 else "f32"
        _close(o, v * result[1], UB[kind] * np.abs(v * result[1]) + 2.0 ** -134, f"tensor {i}")


def test_grad_clip_with_more_chunks_than_the_table_holds(moe):  # noqa: F811
    """A count of another list: the walk ends at the table's last tensor."""
    gen = torch.Generator(device="cuda").manual_seed(34)
    grads = [torch.empty(n, device="cuda").normal_(generator=gen) for n in (7, 5000, 0, 12289)]
    want = [t.clone() for t in grads]
    moe.moe_grad_clip(moe.GradList(want), 0.5)
    for more in (1, 100, 9000):
        mine = [t.clone() for t in grads]
        lst = moe.GradList(mine)
        lst.chunks += more
        lst.ws = torch.empty(2048 * 8, dtype=torch.uint8, device="cuda")
        log(f"moe_grad_clip with {more} chunks too many")
        moe.moe_grad_clip(lst, 0.5)
        for t, w in zip(mine, want):
            assert float((t - w).abs().max()) <= 2.0 ** -22 * float(w.abs().max()) if t.numel() else True
