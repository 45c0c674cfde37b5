"""The decode operators' oracle against properties of its definitions (CPU)."""

import numpy as np
import pytest

from oracle import decode as O


def pool(seed, pages=30, page=4, seqs=8, cols=6):
    rng = np.random.default_rng(seed)
    k = rng.standard_normal((2, pages, 2, page, 3))
    return rng, O.Pool(np.full((seqs, cols), -1), [0] * seqs, [0] * pages, k, -k)


def contents(p, s):
    at = [p.position(s, t) for t in range(p.lens[s])]
    return np.array([[p.k[:, a, :, r], p.v[:, a, :, r]] for a, r in at])


@pytest.mark.parametrize("seed", range(5))
def test_counts_are_the_tables_entries_and_contents_survive(seed):
    rng, p = pool(seed)
    for _ in range(10):
        seq = rng.permutation(8)[:3].tolist()
        p.extend(seq, rng.integers(0, 9, 3).tolist())
        a, b, c = rng.permutation(8)[:3].tolist()
        want = contents(p, a)
        p.fork([a], [b])
        if p.lens[b] == p.lens[a]:
            assert np.array_equal(contents(p, b), want) and np.array_equal(contents(p, a), want)
        else:
            assert p.lens[b] == 0 and p.no_page
        p.free([c])
        held = [e for s, row in enumerate(p.table) for e in row[:p.held(p.lens[s])]]
        assert all(p.refs[e] == held.count(e) for e in range(len(p.refs)))
    before = [contents(p, s) for s in range(8)]
    live = p.compact()
    assert all(p.refs[:live]) and not any(p.refs[live:])
    assert all(np.array_equal(contents(p, s), before[s]) for s in range(8))


def test_an_append_never_meets_a_shared_page():
    rng, p = pool(9)
    p.extend([0], [6])
    p.fork([0, 0], [1, 2])
    for s in range(3):
        p.extend([s], [1])
        page, _ = p.position(s, p.lens[s] - 1)
        assert p.refs[page] == 1


def test_attention_of_a_zero_query_is_the_mean_and_windows_nest():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 9, 2, 4))
    out, lse, _, _ = O.attention(np.zeros((4, 4)), k, v, 0.5)
    assert np.allclose(out[:2], v[:, 0].mean(0)) and np.allclose(out[2:], v[:, 1].mean(0))
    assert np.allclose(lse, np.log(9))
    assert O.visible(9, 0, 0) == O.visible(9, 9, 0) == O.visible(9, 4, 5) == list(range(9))
    assert O.visible(9, 2, 3) == [0, 1, 2, 7, 8] and O.visible(0, 2, 3) == []
    q = rng.standard_normal((4, 4))
    a, la, _, _ = O.attention(q, k[:5], v[:5], 1.0)
    b, lb, _, _ = O.attention(q, k[5:], v[5:], 1.0)
    whole, lw, _, _ = O.attention(q, k, v, 1.0)
    w = np.exp(np.stack([la, lb]) - lw)
    assert np.allclose(w.sum(0), 1) and np.allclose(w[0][:, None] * a + w[1][:, None] * b, whole)


def test_guided_logits_at_scales_zero_and_one_and_their_edges():
    rng = np.random.default_rng(2)
    cond, uncond = rng.standard_normal((2, 50))
    assert np.array_equal(O.guided_logits(cond, uncond, 1.0)[0], cond)
    assert np.allclose(O.guided_logits(cond, uncond, 0.0)[0], uncond)
    z, token, logprob, _, _ = O.guided_logits(cond, uncond, 2.5)
    assert np.allclose(z, uncond + 2.5 * (cond - uncond)) and token == int(z.argmax())
    assert np.isclose(np.exp(z - z[token] + logprob).sum(), 1.0)
    cond[3] = uncond[3] = -np.inf
    uncond[4] = -np.inf
    z = O.guided_logits(cond, uncond, 3.0)[0]
    assert np.isneginf(z[3]) and z[4] == cond[4]
    z, token, logprob, _, _ = O.guided_logits(cond, allowed=np.zeros(50, bool))
    assert token == -1 and np.isneginf(logprob) and np.isneginf(z).all()
    z = O.guided_logits(np.array([2.0, -2.0, 1.0, 1.0]), tokens=[0, 1, 2, 2, 9, -1], prompt=2, repetition=2.0,
                        frequency=0.5, presence=0.25)[0]
    assert np.allclose(z, [1.0, -4.0, 0.5 - 1.25, 1.0])
