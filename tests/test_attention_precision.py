"""How exactly mk_prefix_attention holds its probabilities: one rule for every call.

Each probability enters the product with V as a bf16 value and the bf16 rounding of what that
left out, as in the decode step.  Per element, with u = 2^-8 (half a step of bf16 relative to
the value), n visible keys, A = sum_j p_j |v_j| / sum_j p_j and E the bound on a score's error
of test_prefix_attention.py:

- the result is rounded to bf16: u |exact|;
- p in [1, 2) leaves a rest of at most 2^-8, and that one's rounding is off by at most 2^-17
  (the same relative to p in every binade): 2^-17 A;
- the exponential: 2^-22 for each p and its share of the sum: 2^-20 A with the divisions;
- 2 n products in 32 bits, each chopped by at most 2^-23, and some 64 more sums: (2 n + 64) 2^-23 A;
- the scores move each probability by e^E, and the rounding of the exponential's argument,
  3 * 2^-24 of a score, is less than E / 10 (D >= 32): 2.2 E A.

With few keys the bf16 rounding of p alone is off by up to 2^-8 A, so a lost or misplaced rest
shows where the exact result is small beside A."""
import numpy as np
import pytest

from test_prefix_attention import Case

gpu = pytest.mark.gpu


def bound(c, want):
    eo, _, A, E = want
    n = np.zeros(c.n_tokens)
    for b, L in enumerate(c.lens):
        for t in range(c.T[b]):
            n[int(c.off[b]) + t] = max(0, L - c.T[b] + t + 1)
    rest = 2.0 ** -17 + 2.0 ** -20 + (2.0 * n[:, None] + 64.0) * 2.0 ** -23 + 2.2 * E
    return 2.0 ** -8 * np.abs(eo) + rest[..., None] * A


def worst(c, out=None, want=None):
    want = want or c.exact()
    tol, n = bound(c, want), int(c.off[-1])
    out = c.run()[0] if out is None else out
    return float(np.max((np.abs(out - want[0]) / np.maximum(tol, 1e-30))[:n]))


def small_scores(c):
    """Flat softmaxes: the scores' own error is far below the rounding of p."""
    c.q = (c.q.float() * 0.25).to(c.q.dtype)
    return c


@gpu
@pytest.mark.parametrize("heads", [(16, 4, 64), (32, 4, 128), (6, 2, 32), (4, 4, 64)])
@pytest.mark.parametrize("each", [1, 3, 4, 5, 8, 16])
def test_single_tokens(heads, each):
    """Samples of a short prompt, few results and many."""
    c = small_scores(Case([(32, [(1 + 3 * i % 20, 1) for i in range(each)])], heads, seed=each))
    assert worst(c) <= 1.0


@gpu
@pytest.mark.parametrize("heads", [(16, 4, 64), (32, 4, 128), (6, 2, 32)])
def test_several_tokens_and_pairs_of_row_tiles(heads):
    c = small_scores(Case([(16, [(12, 9), (40, 40), (70, 70)]), (0, [(9, 9), (130, 130)])], heads))
    assert worst(c) <= 1.0


@gpu
@pytest.mark.parametrize("heads", [(8, 1, 64), (64, 1, 128)])
def test_pieces_of_a_split_item(heads):
    """A long sequence over several SMs of which a few scattered keys count: the others' scores
    lie 100 and more below, so that their p are 0 and add no error."""
    c, D = Case([(0, [(4000, 1)])], heads), heads[2]
    at = [3, 130, 700, 701, 1500, 1777, 2200, 2900, 3333, 3999]
    c.q = c.q.abs()
    k = c.k[c.rows[0]].transpose(0, 1).reshape(1, -1, D)
    few = (0.1 * k[:, at].float()).to(c.k.dtype)
    k[:] = -16.0
    k[:, at] = few
    c.k[c.rows[0]] = k.view(1, -1, 16, D).transpose(0, 1).contiguous()
    K, q = few[0].double().numpy(), c.q[0].double().numpy()
    V = c.v[c.rows[0]].transpose(0, 1).reshape(-1, D)[at].double().numpy()
    scale = 1.0 / np.sqrt(D)
    s = q @ K.T * scale
    assert (q.sum(1) * -16.0 * scale < s.min(1) - 100.0).all()
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    E = (np.abs(q) @ np.abs(K).T).max(1) * scale * D * 2.0 ** -23
    rest = 2.0 ** -17 + 2.0 ** -20 + (2.0 * len(at) + 64.0) * 2.0 ** -23 + 2.2 * E
    out = c.run()[0][0]
    assert (np.abs(out - p @ V) <= 2.0 ** -8 * np.abs(p @ V) + rest[:, None] * (p @ np.abs(V))).all()


@gpu
def test_a_batch_is_as_exact_in_a_larger_handle():
    """The rounding of a row depends on neither the other rows nor the handle's capacity."""
    c = small_scores(Case([(32, [(5, 1), (9, 1)])], (16, 4, 64)))
    want = c.exact()
    wide = Case([(32, [(5, 1), (9, 1)])], (16, 4, 64), extra_rows=300)
    t = c.t
    wide.q[:2] = c.q
    wide.q[2:] = 0.0
    out, _ = wide.run(offsets=True)
    assert worst(c, out[:2], want) <= 1.0
    assert bool(t.equal(wide.k, c.k))


def test_the_bound_tells_a_lost_rest():
    """The same sums with p rounded to bf16 alone break the bound (without a GPU)."""
    import torch

    c = small_scores(Case([(32, [(1 + 3 * i % 20, 1) for i in range(5)])], (16, 4, 64), seed=5))
    want = c.exact()
    one, two = np.zeros_like(want[0]), np.zeros_like(want[0])
    k, v, q = (x.double().numpy() for x in (c.k, c.v, c.q))
    for b, L in enumerate(c.lens):
        K = k[c.rows[b]].transpose(1, 0, 2, 3).reshape(c.Hkv, -1, c.D)[:, :L]
        V = v[c.rows[b]].transpose(1, 0, 2, 3).reshape(c.Hkv, -1, c.D)[:, :L]
        for h in range(c.Hq):
            s = K[h // 4] @ q[b, h] / 8.0
            p = torch.from_numpy(np.exp(s - s.max()))
            hi = p.to(torch.bfloat16).double()
            lo = (p - hi).to(torch.bfloat16).double()
            for out, w in ((one, hi), (two, hi + lo)):
                o = torch.from_numpy((w.numpy() @ V[h // 4]) / float(p.sum()))
                out[b, h] = o.to(torch.bfloat16).double().numpy()
    assert worst(c, two, want) <= 1.0 < worst(c, one, want)
