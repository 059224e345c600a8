"""CPU pins of the fp64 scoring oracle: library softmax, closed forms, finite differences."""
import numpy as np
import pytest
import scipy.special
import scipy.stats

from oracle import scoring_oracle as orc


def draw(N, V, T, seed):
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(N, V)) * 3
    tokens = rng.integers(-1, V, size=(N, T))
    return z, tokens, rng.normal(size=(N, T)), rng.normal(size=N)


def test_score_against_scipy():
    z, tokens, _, _ = draw(6, 40, 3, 0)
    logp, ent, m, log_s = orc.score(z, tokens)
    lq = scipy.special.log_softmax(z, axis=1)
    for n in range(6):
        for t in range(3):
            want = lq[n, tokens[n, t]] if tokens[n, t] >= 0 else 0.0
            assert abs(logp[n, t] - want) < 1e-12
        assert abs(ent[n] - scipy.stats.entropy(np.exp(lq[n]))) < 1e-12
    assert np.allclose(m + log_s, scipy.special.logsumexp(z, axis=1), atol=1e-12)


def test_closed_forms():
    z = np.full((3, 16), -np.inf)
    z[1] = 5.0                   # uniform
    z[2, 7] = -2.0               # one token left
    logp, ent, m, log_s = orc.score(z, np.array([[3], [3], [7]]))
    assert logp[0, 0] == -np.inf and ent[0] == 0 and m[0] == -np.inf and log_s[0] == 0
    assert abs(logp[1, 0] + np.log(16)) < 1e-12 and abs(ent[1] - np.log(16)) < 1e-12
    assert logp[2, 0] == 0 and ent[2] == 0
    dz = orc.logits_gradient(z, np.array([[3], [3], [7]]), np.ones((3, 1)), np.ones(3))
    assert np.all(dz[0] == 0)
    assert np.allclose(dz[1], (np.arange(16) == 3) - 1 / 16, atol=1e-12)  # entropy is stationary
    assert np.allclose(dz[2], 0, atol=1e-12)
    ids, lp = orc.alternatives(np.array([[1.0, 4.0, 4.0, -np.inf, 0.0, -0.0]]), 6)
    assert ids.tolist() == [[1, 2, 0, 4, 5, 3]] and lp[0, 5] == -np.inf


@pytest.mark.parametrize("with_entropy", [False, True])
def test_gradients_against_differences(with_entropy):
    N, V, d, T, h = 3, 11, 5, 4, 1e-6
    z, tokens, g, ge = draw(N, V, T, 1)
    ge = ge if with_entropy else None

    def value(logp, ent):
        return (np.where(tokens < 0, 0, g) * logp).sum() + (0 if ge is None else (ge * ent).sum())

    dz = orc.logits_gradient(z, tokens, g, ge)
    for n in range(N):
        for v in range(V):
            up, dn = z.copy(), z.copy()
            up[n, v] += h
            dn[n, v] -= h
            diff = (value(*orc.score(up, tokens)[:2]) - value(*orc.score(dn, tokens)[:2])) / (2 * h)
            assert abs(diff - dz[n, v]) < 1e-7
    rng = np.random.default_rng(2)
    H, W = rng.normal(size=(N, d)), rng.normal(size=(V, d))
    dH, dW = orc.projected_gradients(H, W, tokens, g, ge)
    for A, dA, f in ((H, dH, lambda x: orc.projected(x, W, tokens)), (W, dW, lambda x: orc.projected(H, x, tokens))):
        for i in np.ndindex(A.shape):
            up, dn = A.copy(), A.copy()
            up[i] += h
            dn[i] -= h
            diff = (value(*f(up)[:2]) - value(*f(dn)[:2])) / (2 * h)
            assert abs(diff - dA[i]) < 1e-7
