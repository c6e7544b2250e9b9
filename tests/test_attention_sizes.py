"""mk_prefix_attention at the sizes where it takes other paths, and at random ones.

Bounds as in test_prefix_attention.py (the calls are the same); the sizes lie on both sides
of each limit: 16 (token, kv head) pairs an SM for the join's narrow blocks, 384 sequences or
groups for a turn of the cut, 1024 and 512 for a call."""
import numpy as np
import pytest

import persistent_moe_decode_sm_gb300 as mk
from test_prefix_attention import Case

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("over", [-1, 0, 1, 400])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_join_of_many_tokens(D, over):
    """Shared pages, so that every token has pieces to join, of which some are split."""
    import torch

    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tokens = 16 * sms // 4 + over                      # 4 kv heads
    first, second = tokens // 3, tokens // 5
    rest = tokens - first - second
    c = Case([(320, [(first + 7, first), (second, second)]), (160, [(rest + 100, rest)])], (8, 4, D),
             seed=over + 2)
    assert c.n_tokens == tokens
    c.check()


@gpu
@pytest.mark.parametrize("heads", [(4, 4, 32), (12, 4, 128)])
def test_join_of_many_single_tokens(heads):
    """1024 sequences of one token in groups of 64, one of them empty and one finished."""
    groups = []
    for g in range(16):
        groups.append((16 * (g + 1), [(1 + (5 * i + g) % 40, 1) for i in range(64)]))
    c = Case(groups, heads, seed=3)
    for b in (5, 64):
        c.lens[b] = 0
        c.tables[b] = -1
    c.check()


@gpu
@pytest.mark.parametrize("n", [383, 384, 385, 767, 768, 1023, 1024])
@pytest.mark.parametrize("grouped", [True, False])
def test_many_sequences(n, grouped):
    """A few tokens each, in as many groups as there can be; the last sequences count."""
    rng = np.random.default_rng(n)
    sizes, left = [], n
    while left:
        k = min(left, int(rng.integers(1, 4)) if len(sizes) < 511 else left)
        sizes.append(k)
        left -= k
    groups = [(int(rng.integers(0, 60)), [(int(rng.integers(1, 30)), int(rng.integers(0, 3)))
                                          for _ in range(k)]) for k in sizes]
    groups[-1] = (40, [(20 + i, 2) for i in range(sizes[-1])])
    c = Case(groups, (4, 2, 64), seed=n)
    assert len(c.lens) == n
    c.check(grouped=grouped)


@gpu
def test_as_many_groups_as_there_can_be():
    c = Case([(16 * (g % 3), [(3 + g % 20, 1), (1, 1)]) for g in range(512)], (2, 1, 32))
    c.check()
    a, b = c.attention(c.device())
    t = c.t
    d = {n: t.zeros(1026, 4, dtype=t.int32, device="cuda") for n in ("tables",)}
    lens = t.ones(1025, dtype=t.int32, device="cuda")
    big = a.batch(d["tables"][:1025], lens)
    with pytest.raises(mk.MkError) as e:
        a.run(0, big, t.zeros(1025, 2, 32, dtype=t.bfloat16, device="cuda"),
              t.zeros(1025, 2, 32, dtype=t.bfloat16, device="cuda"))
    assert e.value.code == mk.MK_ERR_BATCH


@gpu
def test_many_blocks_of_few_tokens():
    """64 heads a kv head: a block of two row tiles has 4 tokens, so 700 tokens are 175 blocks."""
    Case([(40, [(700, 700), (3, 90)])], (64, 1, 32)).check()


@gpu
@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    rng = np.random.default_rng(1000 + seed)

    def log(low, high):
        return int(round(np.exp(rng.uniform(np.log(low), np.log(high)))))

    Hkv, G, D = int(rng.integers(1, 5)), int(rng.integers(1, 17)), int(rng.choice([32, 64, 128]))
    P = int(rng.choice([16, 16, 32, 48, 80, 128, 256]))
    groups, tokens = [], 0
    for _ in range(int(rng.integers(1, 5))):
        seqs = []
        for _ in range(log(1, 40)):
            T = 1 if rng.random() < 0.5 else int(rng.integers(0, log(2, 120)))
            T = min(T, max(0, 6000 // (Hkv * G) - tokens))
            seqs.append((log(1, 700) - 1, T))
            tokens += T
        groups.append((log(1, 3000) - 1, seqs))
    groups[0][1].append((5, 1))
    Case(groups, (Hkv * G, Hkv, D), P, seed=seed, extra_rows=int(rng.integers(0, 5))).check()
