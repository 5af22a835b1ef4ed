"""The float64 training oracle against differences of its own forward formulas
and against closed forms (CPU)."""
import numpy as np
import pytest

from oracle import train

EPS = 1e-5


def _numeric(f, x, h=1e-5):
    """Central differences of the scalar f at x (changed in place and restored);
    error about h^2 |f'''| + 1e-16 |f| / h."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        v = x[i]
        x[i] = v + h
        up = f()
        x[i] = v - h
        g[i] = (up - f()) / (2 * h)
        x[i] = v
    return g


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post", [True, False])
def test_block_norm_backward_against_differences(gate, post):
    rng = np.random.default_rng(1)
    T, H, alpha, beta = 3, 5, 0.9, 0.7
    x, b, dr, dh = (rng.standard_normal((T, H)) for _ in range(4))
    w_pre = 1 + 0.2 * rng.standard_normal(H)
    w_post = 1 + 0.2 * rng.standard_normal(H) if post else None
    gv = {"none": None, "channel": rng.standard_normal(H), "token": rng.standard_normal((T, 1)),
          "full": rng.standard_normal((T, H))}[gate]

    def loss():
        r, h, _ = train.block_norm(x, b, w_pre, w_post, gv, alpha, beta, EPS)
        return (r * dr).sum() + (h * dh).sum()

    r, _, _ = train.block_norm(x, b, w_pre, w_post, gv, alpha, beta, EPS)
    got = train.block_norm_backward(r, dr, dh, b, w_pre, w_post, gv, alpha, beta, EPS)
    for name, v in (("dx", x), ("db", b), ("dw_pre", w_pre), ("dw_post", w_post), ("dgate", gv)):
        if v is not None:
            assert np.allclose(got[name], _numeric(loss, v), atol=1e-8, rtol=1e-7), name
        else:
            assert name not in got


def test_block_norm_first_norm_and_unit_rows():
    x = np.array([[3.0, 4.0], [0.0, 0.0]])
    r, h, _ = train.block_norm(x, None, np.ones(2), None, None, 1.0, 1.0, 1e-30)
    assert np.allclose(h[0], np.array([3.0, 4.0]) / np.sqrt(12.5)) and np.all(h[1] == 0)
    assert r is x


def test_grouped_products_against_a_loop_over_rows():
    rng = np.random.default_rng(2)
    off = np.array([0, 2, 2, 5])
    a, b = rng.standard_normal((4, 6)), rng.standard_normal((3, 7, 6))
    index, scale = np.array([3, 0, 1, 1, 2]), rng.standard_normal(5)
    out, _ = train.grouped_gemm(a, b, off, index, scale)
    kn, _ = train.grouped_gemm(a, b.transpose(0, 2, 1), off, index, scale, kn=True)
    dy = rng.standard_normal((5, 7))
    dw, _ = train.grouped_wgrad(dy, a, off, None, index)
    want = np.zeros_like(dw)
    for r, g in enumerate([0, 0, 2, 2, 2]):
        assert np.allclose(out[r], scale[r] * b[g] @ a[index[r]])
        want[g] += np.outer(dy[r], a[index[r]])
    assert np.allclose(out, kn) and np.allclose(dw, want) and np.all(dw[1] == 0)


def test_swiglu_backward_against_differences():
    rng = np.random.default_rng(3)
    a, dh, w = rng.standard_normal((3, 8)), rng.standard_normal((3, 4)), rng.standard_normal(3)
    da, dgate, hg, _ = train.swiglu_backward(a, dh, w)
    loss = lambda: (w[:, None] * train.swiglu(a) * dh).sum()  # noqa: E731
    assert np.allclose(da, _numeric(loss, a), atol=1e-8, rtol=1e-7)
    assert np.allclose(dgate, _numeric(loss, w), atol=1e-8, rtol=1e-7)
    assert np.allclose(hg, w[:, None] * train.swiglu(a))


def test_clip_closed_form():
    norm, coef = train.clip([np.full(16, 0.5), np.array([1.0, 2.0])], 0.6)
    assert norm == 3.0 and abs(coef - 0.6 / 3.000001) < 1e-15
    assert train.clip([np.array([0.3])], 1.0)[1] == 1.0
    assert train.clip([np.array([np.inf])], 1.0)[1] == 1.0
