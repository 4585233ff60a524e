"""Pins of the objectives' float64 oracle (CPU): published vectors of the
generator, gradients against differences of the losses, and the definitions
on inputs small enough to work out."""
import numpy as np
import pytest

from oracle import objectives as O


def test_philox_published_vectors():
    """The generator's known-answer vectors (its authors' test file)."""
    f = 0xFFFFFFFF
    assert O.philox((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert O.philox((f, f, f, f), (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert O.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def differences(loss, x, h=1e-5):
    """Central differences of a scalar function of a matrix; error ~ h^2 f''' / 6 + 1e-16 f / h."""
    g = np.zeros(x.shape)
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = (loss(up) - loss(down)) / (2 * h)
    return g


# differences err by about h^2 + 1e-16 / h ~ 1e-10 of the loss's scale (~ 1 here)
TOL = 1e-8


@pytest.mark.parametrize("kl,s", [(0.0, 1.0), (0.3, 1.0), (0.1, 0.6)])
def test_policy_gradient(kl, s):
    rng = np.random.default_rng(0)
    x = rng.normal(size=(7, 5))
    labels = np.array([0, 4, -1, 2, 2, 1, 3])
    adv, w = rng.normal(size=7), np.array([.1, .2, .3, 0, .1, .2, .1])
    old = O.token_logp(x, labels, s) + 0.3 * rng.normal(size=7)
    ref = O.token_logp(x, labels, s) + 0.3 * rng.normal(size=7)
    run = lambda y: O.policy_loss(y, labels, adv, w, old, ref, 0.2, 0.28, kl, s)
    assert np.abs(run(x)[2] - differences(lambda y: run(y)[0][0], x)).max() < TOL
    assert run(x)[0][3] > 0       # some rows are clipped


@pytest.mark.parametrize("kind,eps,average", [("sigmoid", 0.0, False), ("sigmoid", 0.1, True), ("squared", 0.0, False),
                                              ("squared", 0.0, True)])
def test_preference_gradient(kind, eps, average):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(10, 4))
    labels = np.array([0, 3, -1, 2, 2, 1, 3, 0, 1, 2])
    offsets = [0, 3, 4, 8, 8]          # the last sequence is empty; rows 8 and 9 are in none
    ref, w = rng.normal(size=10) - 1.4, [0.7, 0.4]
    run = lambda y: O.preference_loss(y, labels, offsets, ref, w, 0.5, kind, eps, average)
    assert np.abs(run(x)[3] - differences(lambda y: run(y)[0][0], x)).max() < TOL
    assert not run(x)[3][8:].any()


@pytest.mark.parametrize("z", [0.0, 0.01])
def test_balance_gradient(z):
    rng = np.random.default_rng(2)
    x = rng.normal(size=(6, 5))
    chosen = np.array([[0, 1], [2, -1], [4, 0], [1, 2], [3, 4], [0, 2]])
    mask = np.array([1, 1, 0, 1, 1, 1], bool)
    run = lambda y: O.balance_loss(y, chosen, mask, 0.1, z)
    assert np.abs(run(x)[3] - differences(lambda y: run(y)[0][0], x)).max() < TOL
    stats, counts, prob, grad = run(x)
    assert counts.tolist() == [2, 2, 3, 1, 1] and abs(prob.sum() - 1) < 1e-12 and stats[3] == 5
    assert not grad[2].any()


def test_dropout_keeps_its_share():
    keep = O.dropout_keep(40, 101, 7, 1 << 40, 0.25)
    # 4040 draws: standard deviation of the share is 0.0068
    assert abs(keep.mean() - 0.75) < 5 * 0.0068
    assert O.dropout_keep(2, 9, 1, 0, 0.0).all() and not O.dropout_keep(2, 9, 1, 0, 1.0).any()
    assert (O.dropout_keep(2, 33, 1, 0, 0.5) != O.dropout_keep(2, 33, 1, 1, 0.5)).any()
    assert (O.dropout_keep(2, 33, 1, 0, 0.5) != O.dropout_keep(2, 33, 2, 0, 0.5)).any()
