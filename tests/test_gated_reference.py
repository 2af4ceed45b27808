"""The 64-bit form of the gated products' activations: their slopes against
central differences, and the bounds that the GPU tests take for given."""
import numpy as np
import pytest

import gated_reference as ref


@pytest.mark.parametrize("name", ref.ACTS)
def test_slopes_are_the_differences(name):
    g = np.linspace(-12.0, 12.0, 2001)
    e = 1e-5
    a, s = ref.act(g, name)
    difference = (ref.act(g + e, name)[0] - ref.act(g - e, name)[0]) / (2 * e)
    # third derivatives are below 10: off by at most 10 e^2 / 6, and by 2 roundings of |a| over 2 e
    assert np.all(np.abs(difference - s) <= 10 * e * e / 6 + 4 * 2.0 ** -53 * (np.abs(a) + 1) / e)
    assert np.max(np.abs(s)) <= 1.13
    second = (ref.act(g + e, name)[1] - ref.act(g - e, name)[1]) / (2 * e)
    assert np.max(np.abs(second)) <= 1.13


@pytest.mark.parametrize("name", ref.ACTS)
def test_far_ends(name):
    """Far to the left nothing is left of the activation, far to the right all of g."""
    a, s = ref.act(np.array([-60.0, 60.0]), name)
    assert abs(a[0]) < 1e-20 and a[1] == 60.0 and abs(s[0]) < 1e-20 and s[1] == 1.0


@pytest.mark.parametrize("name", ref.ACTS)
def test_gradients_of_a_small_product(name):
    """The gradients of sum(d h) from the slopes, against differences in every weight and input."""
    rng = np.random.default_rng(1)
    x, w, d = rng.normal(size=(3, 4)), rng.normal(size=(10, 4)), rng.normal(size=(3, 5))
    r = ref.Gated(x, w, name)
    pre = np.concatenate((d * r.by_gate, d * r.by_up), axis=1)
    e = 1e-6
    for grad, at in ((pre @ w, x), (pre.T @ x, w)):
        for i in np.ndindex(at.shape):
            keep, ends = at[i], []
            for v in (keep + e, keep - e):
                at[i] = v
                ends.append(np.sum(d * ref.Gated(x, w, name).h))
            at[i] = keep
            assert abs((ends[0] - ends[1]) / (2 * e) - grad[i]) <= 1e-7 * (1 + abs(grad[i]))
