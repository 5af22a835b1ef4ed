"""GPU parity of the bf16 training operators (block norms, grouped products,
gated activation, gradient clipping) against the float64 oracle
(``oracle.train``).

Bars: an output is a float32 evaluation rounded once.  UB = 2^-8 (bf16) or
2^-24 (float32) bounds the rounding relative to the value; the float32 part is
bounded by a count of roundings times 2^-24 times the sum of the magnitudes of
the terms (which the oracle returns): FLT = 2^-17 covers 128 roundings, more
than any row's chain (16 products per lane, 6 wave steps, 16 waves, the
statistics' square root and division); sums over n terms add n * 2^-24, and the
matrix instructions, whose inner order and rounding are not specified, are
allowed 2^-23 per product."""
import numpy as np
import pytest

import synth
from helpers import bf16_from_dev, bf16_to_dev, log, to_dev
from oracle import train

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FLT = 2.0 ** -17
UB = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
EPS = 1e-6


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a device"
    import fp8_block_scaled_sigmoid_amd as m
    m.lib()
    return m


def _make(rng, shape, kind, scale=1.0, pad=0, offset=0):
    """(device tensor, its float64 values); pad extra columns and an element
    offset make strided, oddly aligned rows."""
    v = (rng.standard_normal(shape) * scale).astype(np.float32)
    if kind == "bf16":
        bits = synth.f32_to_bf16_bits(v)
        t, v = bf16_to_dev(bits), synth.as_f64(bits)
    else:
        t, v = to_dev(v), v.astype(np.float64)
    if pad or offset:
        t = _strided(t, pad, offset)
    return t, v


def _strided(t, pad, offset):
    rows, cols = t.shape
    ld = cols + pad
    buf = torch.full((offset + rows * ld + 8,), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(t)
    return view


def _val(t):
    if t.dtype == torch.bfloat16:
        return synth.as_f64(bf16_from_dev(t))
    return t.cpu().numpy().astype(np.float64)


def _close(got, want, tol, what):
    got = _val(got) if torch.is_tensor(got) else got
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= tol + 1e-37)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst "
                           f"{np.nanmax(np.abs(got - want) / (tol + 1e-37)):.2f} of the bar")


def _offsets(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)


# ---------------------------------------------------------------------------
# block norms

NORM_CASES = [
    # T, H, x, b, gate, post norm, pre norm
    (1, 7168, "bf16", "bf16", "channel", True, True),
    (37, 7168, "bf16", "bf16", "token", True, True),
    (5, 16384, "f32", "f32", "full", True, True),
    (9, 8200, "f32", "bf16", "channel", True, True),
    (33, 2049, "f32", "bf16", "full", True, True),
    (19, 513, "bf16", "f32", "token", True, True),
    (600, 64, "bf16", "bf16", "channel", True, True),
    (301, 1, "f32", "f32", "none", True, True),
    (17, 7, "bf16", "bf16", "full", True, True),
    (40, 256, "bf16", "bf16", "none", False, True),
    (40, 1000, "bf16", "bf16", "token", False, True),
    (12, 1030, "bf16", "bf16", "channel", True, False),
    (700, 1024, "bf16", "bf16", "none", True, True),
]


def _norm_inputs(rng, T, H, xk, bk, gate, post, pre, pad=0, offset=0):
    x = _make(rng, (T, H), xk, 1.0, pad, offset)
    b = _make(rng, (T, H), bk, 0.3, pad, offset)
    w_pre = _make(rng, (H,), "f32") if pre else (None, None)
    w_post = _make(rng, (H,), "f32") if post else (None, None)
    g = {"none": (None, None), "channel": None, "token": None, "full": None}[gate]
    if gate == "channel":
        g = _make(rng, (H,), "f32")
    elif gate == "token":
        g = _make(rng, (T, 1), "f32")
    elif gate == "full":
        g = _make(rng, (T, H), bk, 1.0, pad, offset)
    return x, b, w_pre, w_post, g


@pytest.mark.parametrize("case", NORM_CASES, ids=str)
@pytest.mark.parametrize("strided", [False, True])
def test_block_norm_forward(moe, case, strided):
    T, H, xk, bk, gate, post, pre = case
    rng = np.random.default_rng(T * 31 + H)
    pad, offset = (3, 1) if strided else (0, 0)
    x, b, wq, wp, g = _norm_inputs(rng, T, H, xk, bk, gate, post, pre, pad, offset)
    log(f"moe_block_norm {case} strided={strided}")
    r_out = torch.zeros(T, H + pad, dtype=x[0].dtype, device="cuda")[:, :H]
    r, h = moe.moe_block_norm(x[0], b[0], wq[0], wp[0], g[0], alpha=0.8, beta=0.6, eps=EPS, r=r_out)
    wr, wh, mag = train.block_norm(x[1], b[1], wq[1], wp[1], g[1], np.float32(0.8), np.float32(0.6),
                                   EPS)
    _close(r, wr, UB[xk] * np.abs(wr) + FLT * mag, "r")
    if pre:
        ir = train.inv_rms(wr, EPS)
        tol = UB[bk] * np.abs(wh) + FLT * ir * np.abs(wq[1]) * (
            mag + np.abs(wr) * ir * ir * (np.abs(wr) * mag).mean(1, keepdims=True))
        _close(h, wh, tol + FLT * np.abs(wh), "h")
    else:
        assert h is None


@pytest.mark.parametrize("case", NORM_CASES, ids=str)
@pytest.mark.parametrize("strided", [False, True])
def test_block_norm_backward(moe, case, strided):
    T, H, xk, bk, gate, post, pre = case
    rng = np.random.default_rng(T * 37 + H)
    pad, offset = (5, 3) if strided else (0, 0)
    r, b, wq, wp, g = _norm_inputs(rng, T, H, xk, bk, gate, post, pre, pad, offset)
    dr = _make(rng, (T, H), xk, 0.1, pad, offset)
    dh = _make(rng, (T, H), bk, 0.1, pad, offset) if pre else (None, None)
    log(f"moe_block_norm_backward {case} strided={strided}")
    got = moe.moe_block_norm_backward(r[0], dr[0], dh[0], b[0], wq[0], wp[0], g[0], alpha=0.8,
                                      beta=0.6, eps=EPS)
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


def test_block_norm_first_norm_of_a_model(moe):
    rng = np.random.default_rng(5)
    x, dr, dh, w = (_make(rng, s, k) for s, k in (((21, 1032), "bf16"), ((21, 1032), "bf16"),
                                                  ((21, 1032), "bf16"), ((1032,), "f32")))
    log("moe_block_norm without a block output")
    r, h = moe.moe_block_norm(x[0], None, w[0], eps=EPS)
    assert r is x[0]
    _, wh, mag = train.block_norm(x[1], None, w[1], None, None, 1.0, 1.0, EPS)
    _close(h, wh, (UB["bf16"] + FLT) * np.abs(wh), "h")
    dx, db, dw, dwp, dg = moe.moe_block_norm_backward(x[0], dr[0], dh[0], w_pre=w[0], eps=EPS)
    want = train.block_norm_backward(x[1], dr[1], dh[1], None, w[1], None, None, 1.0, 1.0, EPS)
    assert db is None and dwp is None and dg is None
    _close(dx, want["dx"], UB["bf16"] * np.abs(want["dx"]) + FLT * want["mag"]["dx"], "dx")
    _close(dw, want["dw_pre"], 2 * FLT * want["mag"]["dw_pre"], "dw_pre")
    dx2 = moe.moe_block_norm_backward(x[0], None, dh[0], w_pre=w[0], eps=EPS)[0]
    want = train.block_norm_backward(x[1], None, dh[1], None, w[1], None, None, 1.0, 1.0, EPS)
    _close(dx2, want["dx"], UB["bf16"] * np.abs(want["dx"]) + FLT * want["mag"]["dx"], "dx, dr None")


def test_block_norm_in_place_rows_of_zeros_and_non_finite_rows(moe):
    rng = np.random.default_rng(6)
    T, H = 600, 776
    x, b = _make(rng, (T, H), "bf16"), _make(rng, (T, H), "bf16")
    w = _make(rng, (H,), "f32")[0]
    b[0][3] = 0
    x[0][3] = 0
    log("moe_block_norm rows of zeros, in place, non-finite")
    r0, h0 = moe.moe_block_norm(x[0], b[0], w, w, eps=EPS)
    assert torch.all(r0[3] == 0) and torch.all(h0[3] == 0)
    x2, b2 = x[0].clone(), b[0].clone()
    r1, h1 = moe.moe_block_norm(x2, b2, w, w, eps=EPS, r=x2, h=b2)
    assert torch.equal(r0, r1) and torch.equal(h0, h1)
    x3 = x[0].clone()
    x3[7, 5] = float("nan")
    x3[9, 0] = float("inf")
    r3, h3 = moe.moe_block_norm(x3, b[0], w, w, eps=EPS)
    ok = [t for t in range(T) if t not in (7, 9)]
    assert torch.equal(r3[ok], r0[ok]) and torch.equal(h3[ok], h0[ok])
    assert torch.isnan(r3[7, 5]) and torch.isnan(h3[7]).all() and torch.isinf(r3[9, 0])
    dr, dh = _make(rng, (T, H), "bf16")[0], _make(rng, (T, H), "bf16")[0]
    a = moe.moe_block_norm_backward(r0, dr, dh, b[0], w, w, eps=EPS)
    dr2, dh2 = dr.clone(), dh.clone()
    c = moe.moe_block_norm_backward(r0, dr2, dh2, b[0], w, w, eps=EPS, dx=dr2, db=dh2)
    for u, v in zip(a[:4], c[:4]):
        assert torch.equal(u, v) and torch.isfinite(u.float()).all()


def test_block_norm_no_tokens(moe):
    e = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(128, device="cuda")
    r, h = moe.moe_block_norm(e, e, w, w)
    assert r.shape == h.shape == (0, 128)
    dw = torch.full((128,), 7.0, device="cuda")
    got = moe.moe_block_norm_backward(e, e, e, e, w, w, gate=w, dw_pre=dw)
    for t in got[2:]:
        assert torch.all(t == 0)


# ---------------------------------------------------------------------------
# grouped products

SIZES = {"ragged": [17, 0, 260, 128, 1], "one": [1], "empty ends": [0, 0, 40, 0],
         "single": [333], "many": [3] * 70, "large": [0, 700, 300, 515],
         "small with a long one": [5] * 11 + [0] * 20 + [300] + [33, 64, 97, 128, 2] + [0] * 5,
         "rests": [256, 257, 384, 385, 512, 129, 128, 0, 1000]}
GEMM_CASES = [
    # sizes, n_out, k, kn, gather, scale, out
    ("ragged", 512, 384, False, True, True, "bf16"),
    ("ragged", 384, 512, True, False, False, "f32"),
    ("ragged", 264, 136, False, False, True, "f32"),
    ("ragged", 136, 264, True, True, True, "bf16"),
    ("one", 8, 8, False, False, False, "f32"),
    ("one", 1024, 2048, False, True, False, "bf16"),
    ("one", 1024, 2048, True, True, False, "bf16"),
    ("empty ends", 200, 1000, False, True, False, "f32"),
    ("single", 712, 40, True, False, False, "bf16"),
    ("many", 256, 520, False, True, False, "bf16"),
    ("many", 520, 256, True, True, True, "f32"),
    ("large", 1288, 1096, False, True, True, "bf16"),
    ("large", 1096, 1288, True, True, True, "bf16"),
    ("large", 512, 128, False, False, False, "bf16"),
    ("small with a long one", 1288, 200, False, True, True, "bf16"),
    ("small with a long one", 264, 1032, True, False, False, "f32"),
    ("small with a long one", 24, 64, True, True, False, "bf16"),
    ("rests", 520, 456, False, True, False, "bf16"),
    ("rests", 776, 136, True, False, True, "f32"),
    ("rests", 256, 8, False, False, False, "f32"),
]


@pytest.mark.parametrize("case", GEMM_CASES, ids=str)
def test_grouped_gemm_bf16(moe, case):
    name, n, k, kn, gather, scale, out = case
    sizes = SIZES[name]
    off = _offsets(sizes)
    R, G = int(off[-1]), len(sizes)
    rng = np.random.default_rng(n + k)
    src = 97 if gather else R + 2
    a = _make(rng, (src, k), "bf16", pad=8 if gather else 16)
    b = _make(rng, (G, k, n) if kn else (G, n, k), "bf16", 0.1)
    index = rng.integers(0, src, R).astype(np.int32) if gather else None
    s = rng.standard_normal(R).astype(np.float32) if scale else None
    odt = torch.bfloat16 if out == "bf16" else torch.float32
    o = torch.full((R, n + 8), 5.0, dtype=odt, device="cuda")
    log(f"moe_grouped_gemm_bf16 {case}")
    moe.moe_grouped_gemm_bf16(a[0], b[0], to_dev(off), R, b_kn=kn,
                              a_row_index=to_dev(index) if gather else None,
                              row_scale=to_dev(s) if scale else None, out=o[:, :n])
    want, mag = train.grouped_gemm(a[1], b[1], off, index, s, kn)
    _close(o[:, :n], want, UB[out] * np.abs(want) + (k + 8) * 2.0 ** -23 * mag, "out")
    assert torch.all(o[:, n:] == 5.0)


@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("k", [24, 64, 328])
def test_grouped_gemm_bf16_row_tiles(moe, kn, gather, k):
    """Groups at the edges of the row tiles (multiples of 32 rows up to 288),
    each between groups whose rows are not finite."""
    sizes = []
    for r in (257, 288, 289, 576, 577, 600, 864, 865, 1153, 161, 287, 32, 33):
        sizes += [r, 1]
    off = _offsets(sizes)
    R, G, n = int(off[-1]), len(sizes), 520
    rng = np.random.default_rng(k)
    a, b = _make(rng, (R, k), "bf16"), _make(rng, (G, k, n) if kn else (G, n, k), "bf16", 0.1)
    poison = off[1:-1:2]                    # the single rows between
    index = np.arange(R, dtype=np.int32)
    if gather:
        index = rng.permutation(R).astype(np.int32)
    rows = a[0].clone()
    rows[torch.from_numpy(index[poison].astype(np.int64)).cuda()] = float("nan")
    log(f"moe_grouped_gemm_bf16 row tiles, kn {kn}, gather {gather}, k {k}")
    got = moe.moe_grouped_gemm_bf16(rows, b[0], to_dev(off), R, b_kn=kn,
                                    a_row_index=to_dev(index) if gather else None,
                                    out_dtype=torch.float32)
    want, mag = train.grouped_gemm(a[1], b[1], off, index if gather else None, None, kn)
    ok = np.setdiff1d(np.arange(R), poison)
    at = torch.from_numpy(ok).cuda()
    _close(got[at], want[ok], UB["f32"] * np.abs(want[ok]) + (k + 8) * 2.0 ** -23 * mag[ok], "out")
    assert torch.isnan(got[torch.from_numpy(poison.astype(np.int64)).cuda()]).all()


def test_grouped_gemm_bf16_keeps_non_finite_rows_apart(moe):
    rng = np.random.default_rng(8)
    sizes = [5, 130, 0, 9]
    off = _offsets(sizes)
    R, n, k = int(off[-1]), 264, 200
    a, b = _make(rng, (R, k), "bf16"), _make(rng, (4, n, k), "bf16")
    log("moe_grouped_gemm_bf16 / wgrad with non-finite rows")
    clean = moe.moe_grouped_gemm_bf16(a[0], b[0], to_dev(off), R)
    a2 = a[0].clone()
    a2[4] = float("nan")
    a2[135, 7] = float("inf")
    got = moe.moe_grouped_gemm_bf16(a2, b[0], to_dev(off), R)
    ok = [r for r in range(R) if r not in (4, 135)]
    assert torch.equal(got[ok], clean[ok]) and torch.isnan(got[4]).all()
    dy = _make(rng, (R, n), "bf16")[0]
    c = moe.moe_grouped_wgrad_bf16(dy, a[0], to_dev(off), R)
    d = moe.moe_grouped_wgrad_bf16(dy, a2, to_dev(off), R)
    assert torch.equal(c[1:3], d[1:3]) and torch.isnan(d[0]).all()
    bad = [4] + list(range(135, 144))       # another group's rows do not reach group 1
    dy2 = dy.clone()
    dy2[bad] = float("nan")
    e = moe.moe_grouped_wgrad_bf16(dy2, a2, to_dev(off), R)
    assert torch.equal(e[1:3], c[1:3])


WGRAD_CASES = [
    # sizes, n, k, gather a, gather b, out, accumulate
    ("ragged", 512, 384, False, True, "f32", False),
    ("ragged", 264, 136, True, False, "bf16", False),
    ("one", 8, 8, False, False, "f32", False),
    ("empty ends", 200, 1000, True, True, "f32", True),
    ("single", 256, 712, False, False, "f32", False),
    ("many", 256, 136, False, True, "bf16", True),
    ("large", 1288, 1096, False, True, "f32", False),
    ("large", 512, 264, False, False, "f32", True),
    ("rests", 520, 264, True, True, "f32", False),
    ("small with a long one", 136, 520, True, False, "bf16", False),
]


@pytest.mark.parametrize("case", WGRAD_CASES, ids=str)
def test_grouped_wgrad_bf16(moe, case):
    name, n, k, ga, gb, out, accumulate = case
    sizes = SIZES[name]
    off = _offsets(sizes)
    R, G = int(off[-1]), len(sizes)
    rng = np.random.default_rng(n * 3 + k)
    a = _make(rng, (61 if ga else R, n), "bf16", pad=8)
    b = _make(rng, (45 if gb else R, k), "bf16", pad=16)
    ia = rng.integers(0, 61, R).astype(np.int32) if ga else None
    ib = rng.integers(0, 45, R).astype(np.int32) if gb else None
    old = _make(rng, (G, n, k), out)
    log(f"moe_grouped_wgrad_bf16 {case}")
    got = moe.moe_grouped_wgrad_bf16(a[0], b[0], to_dev(off), R,
                                     a_row_index=to_dev(ia) if ga else None,
                                     b_row_index=to_dev(ib) if gb else None,
                                     accumulate=accumulate, out=old[0].clone())
    want, mag = train.grouped_wgrad(a[1], b[1], off, ia, ib)
    if accumulate:
        want, mag = want + old[1], mag + np.abs(old[1])
    _close(got, want, UB[out] * np.abs(want) + (max(sizes) + 8) * 2.0 ** -23 * mag, "dW")


def test_grouped_wgrad_bf16_many_tiles(moe):
    """More tiles than compute units hold at once, of groups with none to many
    steps, gathered on both sides."""
    rng = np.random.default_rng(12)
    sizes = [1, 70, 0, 200, 333, 64, 65, 0, 128, 5, 257, 90, 31, 0, 190, 12] * 2
    off = _offsets(sizes)
    R, n, k = int(off[-1]), 1032, 1544
    a, b = _make(rng, (150, n), "bf16"), _make(rng, (140, k), "bf16")
    ia, ib = (rng.integers(0, m, R).astype(np.int32) for m in (150, 140))
    want, mag = train.grouped_wgrad(a[1], b[1], off, ia, ib)
    log("moe_grouped_wgrad_bf16 many tiles")
    for out in ("f32", "bf16"):
        dt = torch.float32 if out == "f32" else torch.bfloat16
        got = moe.moe_grouped_wgrad_bf16(a[0], b[0], to_dev(off), R, to_dev(ia), to_dev(ib),
                                         out_dtype=dt)
        _close(got, want, UB[out] * np.abs(want) + (max(sizes) + 8) * 2.0 ** -23 * mag, out)
    again = moe.moe_grouped_wgrad_bf16(a[0], b[0], to_dev(off), R, to_dev(ia), to_dev(ib),
                                       out_dtype=torch.bfloat16)
    assert torch.equal(got, again)


def test_grouped_wgrad_bf16_long_single_group_is_deterministic(moe):
    rng = np.random.default_rng(11)
    R, n, k = 5000, 64, 136
    a, b = _make(rng, (R, n), "bf16"), _make(rng, (R, k), "bf16")
    off = to_dev(_offsets([R]))
    log("moe_grouped_wgrad_bf16 5000 rows of one group")
    got = moe.moe_grouped_wgrad_bf16(a[0], b[0], off, R)
    again = moe.moe_grouped_wgrad_bf16(a[0], b[0], off, R)
    assert torch.equal(got, again)
    want, mag = train.grouped_wgrad(a[1], b[1], [0, R])
    _close(got, want, UB["f32"] * np.abs(want) + (R + 8) * 2.0 ** -23 * mag, "dW")
    old = _make(rng, (1, n, k), "bf16")
    got = moe.moe_grouped_wgrad_bf16(a[0], b[0], off, R, accumulate=True, out=old[0].clone())
    want, mag = want + old[1], mag + np.abs(old[1])
    _close(got, want, UB["bf16"] * np.abs(want) + (R + 8) * 2.0 ** -23 * mag, "dW, added")
    off2 = _offsets([2100, 0, 2900])        # two parts a group, one group without rows
    ia = rng.integers(0, R, R).astype(np.int32)
    got = moe.moe_grouped_wgrad_bf16(a[0], b[0], to_dev(off2), R, a_row_index=to_dev(ia))
    want, mag = train.grouped_wgrad(a[1], b[1], off2, ia)
    _close(got, want, UB["f32"] * np.abs(want) + (R + 8) * 2.0 ** -23 * mag, "dW, ragged parts")


# ---------------------------------------------------------------------------
# gated activation


@pytest.mark.parametrize("R,I,kind,pad", [(9, 2048, "bf16", 0), (1, 1, "f32", 0), (5, 7, "bf16", 3),
                                          (300, 129, "f32", 1), (4099, 64, "bf16", 0),
                                          (8200, 40, "bf16", 5), (3, 2056, "f32", 0)])
def test_swiglu_forward_and_backward(moe, R, I, kind, pad):
    rng = np.random.default_rng(R + I)
    a = _make(rng, (R, 2 * I), kind, 2.0, pad, pad)
    dh = _make(rng, (R, I), kind, 0.5, pad, pad)
    w = rng.uniform(0, 1, R).astype(np.float32)
    log(f"moe_swiglu R={R} I={I} {kind} pad={pad}")
    h = moe.moe_swiglu(a[0])
    want = train.swiglu(a[1])
    _close(h, want, (UB[kind] + FLT) * np.abs(want), "h")
    da, dgate, hg = moe.moe_swiglu_backward(a[0], dh[0], to_dev(w))
    wda, wdg, whg, mag = train.swiglu_backward(a[1], dh[1], w)
    # silu' = s + silu (1 - s) cancels near its zero: the float part is
    # relative to the two terms, whose sum is below 1.3
    g, u = a[1][:, :I], a[1][:, I:]
    s = train.sigmoid(g)
    terms = np.abs(w[:, None] * dh[1]) * np.concatenate(
        [np.abs(u) * (s + np.abs(g * s) * (1 - s)), np.abs(g * s)], 1).reshape(R, 2, I).transpose(
            1, 0, 2)
    tol = UB[kind] * np.abs(wda) + FLT * np.concatenate([terms[0], terms[1]], 1)
    _close(da, wda, tol, "da")
    _close(dgate, wdg, FLT * mag + I * 2.0 ** -24 * mag, "dgate")
    _close(hg, whg, (UB[kind] + FLT) * np.abs(whg), "hg")
    da2, none, none2 = moe.moe_swiglu_backward(a[0], dh[0], None, dgate=False, hg=False)
    wda2 = train.swiglu_backward(a[1], dh[1])[0]
    wt = np.maximum(w, 1e-30)[:, None]
    _close(da2, wda2, tol / wt + UB[kind] * np.abs(wda2), "da without a row gate")
    assert none is None and none2 is None


def test_swiglu_extremes(moe):
    v = torch.tensor([[-1e4, -200.0, -89.0, 0.0, 89.0, 1e4, 1.0, 1.0]], device="cuda")
    a = torch.cat([v, torch.ones_like(v)], 1)
    h = moe.moe_swiglu(a)
    assert torch.isfinite(h).all() and torch.all(h[0, :2] == 0) and h[0, 5] == 1e4
    da, dg, hg = moe.moe_swiglu_backward(a, torch.ones_like(v))
    assert torch.isfinite(da).all() and da[0, 0] == 0 and da[0, 5] == 1.0 and da[0, 3] == 0.5
    assert moe.moe_swiglu(torch.empty(0, 16, device="cuda")).shape == (0, 8)


# ---------------------------------------------------------------------------
# gradient norm and clipping


def _grads(rng, spec):
    return [_make(rng, (n,), kind, 0.1) for n, kind in spec]


SPECS = {"one": [(1, "f32")], "mixed": [(5, "bf16"), (16384, "f32"), (16385, "bf16"), (3, "f32"),
                                        (100001, "bf16")],
         "empties": [(0, "f32"), (7, "f32"), (0, "bf16"), (0, "f32")],
         "many": [(1 + 37 * i % 1000, "f32") for i in range(300)]}


@pytest.mark.parametrize("spec", list(SPECS))
@pytest.mark.parametrize("max_norm", [0.05, 1e6, 0.0])
@pytest.mark.parametrize("in_place", [True, False])
def test_grad_clip(moe, spec, max_norm, in_place):
    rng = np.random.default_rng(13)
    grads = _grads(rng, SPECS[spec])
    norm, coef = train.clip([v for _, v in grads], max_norm)
    outs = None
    if not in_place:        # into the other type, at odd addresses of one buffer
        flat = {k: torch.zeros(sum(n for n, _ in SPECS[spec]) + 400, dtype=d, device="cuda")
                for k, d in (("bf16", torch.bfloat16), ("f32", torch.float32))}
        outs, at = [], 1
        for n, kind in SPECS[spec]:
            outs.append(flat["f32" if kind == "bf16" else "bf16"][at:at + n])
            at += n
    log(f"moe_grad_clip {spec} max_norm={max_norm} in_place={in_place}")
    before = [t.clone() for t, _ in grads]
    lst = moe.GradList([t for t, _ in grads], outs)
    sumsq, n32 = moe.moe_grad_norm(lst)
    # squares of 24-bit values are exact in double; 1e-12 covers the sum's order
    assert abs(float(sumsq[0]) - norm ** 2) <= 1e-12 * norm ** 2
    assert abs(float(n32[0]) - norm) <= 2.0 ** -24 * norm + 1e-12 * norm
    result = moe.moe_grad_clip(lst, max_norm).cpu().numpy().astype(np.float64)
    assert abs(result[0] - norm) <= 2.0 ** -23 * norm
    assert abs(result[1] - coef) <= 2.0 ** -21 * coef
    for (t, v), b, o in zip(grads, before, outs or [t for t, _ in grads]):
        if not in_place:
            assert torch.equal(t, b)
        kind = "bf16" if o.dtype == torch.bfloat16 else "f32"
        _close(o, v * result[1], UB[kind] * np.abs(v * result[1]) + 2.0 ** -134, "clipped")
    if in_place and coef == 1.0:
        assert all(torch.equal(t, b) for (t, _), b in zip(grads, before))


def test_grad_clip_extremes(moe):
    big = torch.full((1000,), 1e30, device="cuda")      # its square overflows float
    tiny = torch.full((70000,), 1e-30, device="cuda")   # its square vanishes in float
    lst = moe.GradList([big])
    assert abs(float(moe.moe_grad_norm(lst)[1][0]) / (1e30 * np.sqrt(1000)) - 1) < 1e-6
    lst = moe.GradList([tiny])
    assert abs(float(moe.moe_grad_norm(lst)[1][0]) / (1e-30 * np.sqrt(70000)) - 1) < 1e-6
    for bad in (float("nan"), float("inf")):
        t = torch.ones(100, device="cuda")
        t[50] = bad
        u = torch.ones(7, device="cuda")
        result = moe.moe_grad_clip(moe.GradList([t, u]), 0.5)
        assert not torch.isfinite(result[0]) and result[1] == 1.0
        assert torch.all(u == 1.0) and torch.all(t[:50] == 1.0)


def test_grad_scale_from_a_summed_norm(moe):
    rng = np.random.default_rng(14)
    grads = _grads(rng, SPECS["mixed"])
    lst = moe.GradList([t for t, _ in grads])
    sumsq, _ = moe.moe_grad_norm(lst)
    result = moe.moe_grad_scale(lst, sumsq * 4.0, 0.5)    # as if four ranks held the same
    norm = 2.0 * train.clip([v for _, v in grads], 1.0)[0]
    assert abs(float(result[0]) - norm) <= 2.0 ** -22 * norm
    for t, v in grads:
        w = v * float(result[1])
        _close(t, w, UB["bf16"] * np.abs(w), "scaled")


def test_grad_list_takes_permuted_tensors_and_refuses_others(moe):
    t = torch.ones(6, 8, device="cuda")
    lst = moe.GradList([t.t()])
    moe.moe_grad_clip(lst, 1.0)
    assert abs(float(t.square().sum().sqrt()) - 1.0) < 1e-5
    with pytest.raises(ValueError, match="dense"):
        moe.GradList([t[:, :4]])
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        moe.GradList([t.half()])
    with pytest.raises(ValueError, match="outs"):
        moe.GradList([t], [torch.ones(8, 6, device="cuda")])
    with pytest.raises(moe.MoeError, match="UNSUPPORTED"):
        moe.GradList([t, t])
    with pytest.raises(moe.MoeError, match="UNSUPPORTED"):
        moe.GradList([t.view(-1)[:30], t.view(-1)[29:]])
    with pytest.raises(ValueError, match="at least one"):
        moe.GradList([])


# ---------------------------------------------------------------------------
# refusals of the binding, another stream


def test_refusals(moe):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    off = to_dev(_offsets([4]))
    with pytest.raises(ValueError, match="contiguous rows"):
        moe.moe_block_norm(bf(16, 4).t(), w_pre=torch.ones(16, device="cuda"))
    with pytest.raises(moe.MoeError, match="SHAPE"):
        moe.moe_block_norm(bf(2, 16392), w_pre=torch.ones(16392, device="cuda"))
    with pytest.raises(moe.MoeError, match="SHAPE"):
        moe.moe_block_norm(bf(2, 16), w_pre=torch.ones(16, device="cuda"), eps=0.0)
    with pytest.raises(moe.MoeError, match="NULL"):
        moe.moe_block_norm(bf(2, 16))
    with pytest.raises(ValueError, match="w_pre"):
        moe.moe_block_norm(bf(2, 16), w_pre=torch.ones(15, device="cuda"))
    with pytest.raises(ValueError, match="gate"):
        moe.moe_block_norm(bf(2, 16), bf(2, 16), gate=bf(16))
    with pytest.raises(moe.MoeError, match="NULL"):
        moe.moe_block_norm_backward(bf(2, 16))
    with pytest.raises(moe.MoeError, match="SHAPE"):
        moe.moe_grouped_gemm_bf16(bf(4, 12), bf(1, 8, 12), off, 4)
    with pytest.raises(moe.MoeError, match="SHAPE"):
        moe.moe_grouped_gemm_bf16(bf(3, 16), bf(1, 8, 16), off, 4)
    with pytest.raises(moe.MoeError, match="ALIGN"):
        moe.moe_grouped_gemm_bf16(bf(65)[1:].view(4, 16), bf(1, 8, 16), off, 4)
    with pytest.raises(ValueError, match="group_offsets"):
        moe.moe_grouped_gemm_bf16(bf(4, 16), bf(2, 8, 16), off, 4)
    with pytest.raises(ValueError, match="out"):
        moe.moe_grouped_gemm_bf16(bf(4, 16), bf(1, 8, 16), off, 4, out=bf(4, 16))
    with pytest.raises(moe.MoeError, match="SHAPE"):
        moe.moe_grouped_wgrad_bf16(bf(4, 12), bf(4, 16), off, 4)
    with pytest.raises(ValueError, match="accumulate"):
        moe.moe_grouped_wgrad_bf16(bf(4, 16), bf(4, 16), off, 4, accumulate=True)
    with pytest.raises(ValueError, match="even"):
        moe.moe_swiglu(bf(4, 15))
    with pytest.raises(ValueError, match="dh"):
        moe.moe_swiglu_backward(bf(4, 16), torch.zeros(4, 8, device="cuda"))
    with pytest.raises(moe.MoeError, match="SHAPE"):
        moe.moe_grad_clip(moe.GradList([bf(4)]), -1.0)


@pytest.mark.parametrize("H,T", [(8, (8 << 20) + 5), (2056, (1 << 20) + 7)])
def test_block_norm_more_rows_than_a_launch_holds(moe, H, T):
    """Rows past the first round of the grid: the same bits as in a small call."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.empty(T, H, device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
    w = torch.empty(H, device="cuda").normal_(generator=gen)
    log(f"moe_block_norm {T} x {H}")
    h = moe.moe_block_norm(x, w_pre=w)[1]
    for rows in (slice(0, 9), slice(T - 300, T)):
        assert torch.equal(h[rows], moe.moe_block_norm(x[rows], w_pre=w)[1])


def test_swiglu_backward_more_rows_than_a_launch_holds(moe):
    R, I = (16 << 20) + 11, 8
    gen = torch.Generator(device="cuda").manual_seed(5)
    a = torch.empty(R, 2 * I, device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
    dh = torch.empty(R, I, device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
    g = torch.rand(R, device="cuda", generator=gen)
    log(f"moe_swiglu_backward {R} x {I}")
    got = moe.moe_swiglu_backward(a, dh, g)
    for rows in (slice(0, 9), slice(R - 300, R)):
        for x, y in zip(got, moe.moe_swiglu_backward(a[rows], dh[rows], g[rows])):
            assert torch.equal(x[rows], y)


def test_on_another_stream(moe):
    rng = np.random.default_rng(15)
    x, b = _make(rng, (64, 512), "bf16")[0], _make(rng, (64, 512), "bf16")[0]
    w = torch.ones(512, device="cuda")
    r0, h0 = moe.moe_block_norm(x, b, w, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    log("moe_block_norm on another stream")
    with torch.cuda.stream(s):
        r, h = moe.moe_block_norm(x, b, w, w)
    r2, h2 = torch.empty_like(x), torch.empty_like(x)
    torch.cuda.synchronize()
    moe.moe_block_norm(x, b, w, w, r=r2, h=h2, stream=s)
    s.synchronize()
    assert torch.equal(r, r0) and torch.equal(h, h0) and torch.equal(r2, r0) and torch.equal(h2, h0)
