"""The 64-bit gradients that the GPU tests compare with, against differences of the 64-bit forward
definitions (CPU only)."""
import numpy as np
import pytest

import block_reference as ref


def difference(f, x, h=1e-6):
    """The gradient of the scalar f at x by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        g[i] = (up - f()) / (2 * h)
        x[i] = keep
    return g


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_block_norm_gradients(post, gate):
    rng = np.random.default_rng(1)
    T, H, scale, eps = 3, 7, 0.7, 1e-3
    r, y, d_out, d_new = (rng.standard_normal((T, H)) for _ in range(4))
    w, pw = rng.standard_normal(H), rng.standard_normal(H) if post else None
    f = {"none": None, "channel": rng.standard_normal(H), "token": rng.standard_normal((T, H))}[gate]

    def loss():
        new, _, out, _ = ref.block_norm(r, y, post, pw, f, scale, w, eps)
        return (new * d_new).sum() + (out * d_out).sum()

    new = ref.block_norm(r, y, post, pw, f, scale, w, eps)[0]
    got = ref.block_norm_backward(d_out, d_new, new, y, post, pw, f, scale, w, eps)
    inputs = {"d_residual": r, "d_y": y, "d_weight": w}
    if post:
        inputs["d_post_weight"] = pw
    if f is not None:
        inputs["d_gate"] = f
    assert set(got) == set(inputs)
    for name, x in inputs.items():
        assert np.allclose(got[name][0], difference(loss, x), rtol=1e-6, atol=1e-7), name


@pytest.mark.parametrize("a", ref.ACTIVATIONS)
def test_slopes(a):
    v = np.linspace(-7, 7, 150)   # no point at relu's corner
    assert np.allclose(ref.slope(v, a), (ref.act(v + 1e-6, a) - ref.act(v - 1e-6, a)) / 2e-6, atol=1e-8)
    assert np.abs(ref.slope(np.linspace(-9, 9, 10001), a)).max() <= ref.STEEPEST
