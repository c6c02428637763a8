"""The 64-bit forms that the GPU tests of the mixture-of-experts operators
compare against: their gradients against central differences, and the plan's
rules on its own terms.  CPU only."""
import numpy as np
import pytest

import moe_reference as R


def _differences(f, v, h=1e-5):
    """Central differences of the scalar f at v."""
    g = np.empty_like(v)
    it = np.nditer(v, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = v[i]
        v[i] = old + h
        up = f()
        v[i] = old - h
        down = f()
        v[i] = old
        g[i] = (up - down) / (2 * h)
    return g


@pytest.mark.parametrize("gate", ["none", "channel", "row"])
@pytest.mark.parametrize("parts", ["both", "first", "last"])
def test_norm_gradient_against_differences(gate, parts):
    rng = np.random.default_rng(3)
    T, D = 3, 16
    x, z = rng.normal(size=(T, D)), rng.normal(size=(T, D))
    w_post, w_pre = rng.normal(size=D) + 1, rng.normal(size=D) + 1
    g = {"none": None, "channel": rng.normal(size=D), "row": rng.normal(size=(T, 1))}[gate]
    if parts == "first":
        z = w_post = g = None
    if parts == "last":
        w_pre = None
    dy = rng.normal(size=(T, D))
    dh = rng.normal(size=(T, D)) if w_pre is not None else None
    args = (1e-3, 0.8, 0.6)

    def loss():
        y, h, _, _ = R.norm_fwd(x, z, w_post, g, w_pre, *args)
        return (dy * y).sum() + (0.0 if h is None else (dh * h).sum())

    got = R.norm_bwd(dy, dh, x, z, w_post, g, w_pre, *args)
    for name, v in (("dx", x), ("dz", z), ("dw_post", w_post), ("dgate", g), ("dw_pre", w_pre)):
        assert (name in got) == (v is not None)
        if v is not None:
            # differences: h^2 times third derivatives (below 1e3 here) plus 1e-16 / h
            np.testing.assert_allclose(got[name][0], _differences(loss, v), rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("chosen", [True, False])
def test_route_gradient_against_differences(chosen):
    rng = np.random.default_rng(4)
    T, E, top = 4, 7, 3
    x = rng.normal(size=(T, E))
    x[1, :5] = -np.inf       # two experts left for three slots
    x[2] = -np.inf           # none left
    dw = rng.normal(size=(T, top))
    r = R.route(x, top, chosen)
    assert r["expert"][1, 2] == -1 and (r["expert"][2] == -1).all()
    live = np.isfinite(x)

    def loss():
        return (R.route(x, top, chosen)["weight"] * dw).sum()

    got, _ = R.route_bwd(r, dw, chosen)
    want = np.zeros_like(x)
    for i in np.argwhere(live):
        i = tuple(i)
        old = x[i]
        x[i] = old + 1e-6
        up = loss()
        x[i] = old - 1e-6
        want[i] = (up - loss()) / 2e-6
        x[i] = old
    np.testing.assert_allclose(got, want, rtol=1e-6, atol=1e-7)


def test_plan_orders_the_slots_by_expert():
    x = np.array([[1., 3., 3.], [2., 2., 0.], [-np.inf, 0., 5.], [-np.inf] * 3], dtype=np.float32)
    r = R.route(x, 2, True)
    assert r["expert"].tolist() == [[1, 2], [0, 1], [2, 1], [-1, -1]]  # ties: lowest index
    assert r["sizes"].tolist() == [1, 3, 2] and r["offsets"].tolist() == [0, 128, 256, 384]
    assert r["row"].tolist() == [[128, 256], [0, 129], [257, 130], [-1, -1]]
    assert r["source"][[0, 1, 128, 129, 130, 131, 256, 257, 258]].tolist() == [
        2, -1, 0, 3, 5, -1, 1, 4, -1]
    assert r["source"].size == (8 + 127 * 3) // 128 * 128
