"""Which kernel a routed batch takes, restated from its sizes, and a list of sizes that reaches
every one of them: its layout of a token over lanes, one CTA or many, and the k best one after the
other or by rank.  tests/test_gpu_v_route_layouts.py runs the list."""
import random

# tokens, experts, k
SHAPES = [
    # one CTA
    (1, 8, 1), (3, 8, 2), (9, 16, 2), (20, 5, 4), (20, 32, 4), (11, 8, 8), (30, 64, 3), (30, 64, 8),
    (8, 128, 2), (8, 128, 8), (40, 100, 12), (7, 16, 16), (6, 256, 2), (20, 256, 8), (10, 200, 20),
    (4, 384, 3), (20, 384, 8), (9, 300, 32), (5, 1000, 2), (9, 1000, 8), (6, 1024, 32),
    # many
    (3000, 8, 2), (3000, 5, 5), (3000, 16, 6), (9000, 32, 4), (2000, 64, 3), (5000, 64, 8), (2000, 128, 2),
    (2000, 128, 8), (3000, 70, 5), (2000, 256, 3), (2000, 256, 8), (1500, 384, 2), (2000, 384, 8), (1000, 512, 6),
    (500, 100, 12), (900, 20, 16), (600, 256, 9), (700, 129, 32), (400, 500, 17), (500, 1000, 3), (500, 1000, 8),
    (300, 1024, 32)]


def many_lanes(E, k):
    lanes = 1
    while lanes < 32 and (lanes * 8 < E or lanes < k):
        lanes *= 2
    return lanes, 32 if E > 512 else (16 if E > 256 else 8), 1


def few_lanes(E):
    for most, shape in ((8, (1, 8, 8)), (16, (1, 16, 8)), (32, (2, 16, 4)), (64, (4, 16, 2)),
                        (128, (4, 32, 2)), (256, (8, 32, 1))):
        if E <= most:
            return shape
    return 16, 32, 1


def threads_of(lpt, vpl, one):
    return 256 if (lpt, vpl) == (32, 32) else (512 if one or vpl > 8 or lpt == 1 else 1024)


def forward(T, E, k):
    """(lanes a token, columns a lane, choices a lane, one CTA, chosen by rank)"""
    s = many_lanes(E, k)
    one = T <= 2 * (threads_of(s[0], s[1], True) // s[0]) and T * k <= 4096
    if not one and k <= 8 and E <= 512:
        s = few_lanes(E)
    lpt, _, kpl = s
    rank = (lpt >= 8 or (lpt == 4 and kpl > 1)) and k > 3 and (lpt == 32 or k <= 8)
    return (*s, one, rank)


def backward(E, k):
    if k <= 8 and E <= 256:
        return next(s for most, s in ((8, (1, 8, 8)), (16, (1, 16, 8)), (32, (2, 16, 4)), (64, (4, 16, 2)),
                                      (128, (8, 16, 1)), (256, (16, 16, 1))) if E <= most)
    return many_lanes(E, k)


def test_the_list_reaches_every_kernel():
    rng = random.Random(1)
    sizes = [(T, E, k) for E in range(1, 1025) for k in range(1, min(E, 32) + 1)
             for T in (1, rng.randint(1, 300), 1 << 20)]
    ahead, back = {forward(*s) for s in sizes}, {backward(E, k) for _, E, k in sizes}
    assert len(ahead) > 25 and len(back) == 10
    assert ahead - {forward(*s) for s in SHAPES} == set()
    assert back - {backward(E, k) for _, E, k in SHAPES} == set()


# ------------------------------------------------------------------ candidates of a choice by rank
MOST = 31  # that are ranked; with more, one after the other


def parts_of(lpt, vpl):
    """The part of each column of a token: 16 of them (32 where a token has a warp), whose maxima
    bound the k-th best from below."""
    n = 16 // lpt if lpt < 16 else 1  # of a lane
    run = 8 if n <= vpl // 8 else 4
    part = []
    for c in range(lpt * vpl):
        lane, i = c // 8 % lpt, c // (8 * lpt) * 8 + c % 8
        part.append(lane * n + i // run % n)
    return part


def candidates(row, lpt, vpl, k):
    """How many of a row of distinct logits are not below that bound."""
    best = {}
    for v, p in zip(row, parts_of(lpt, vpl)):
        best[p] = max(v, best.get(p, v))
    parts = 32 if lpt == 32 else 16
    tops = sorted(best.values(), reverse=True) + [float("-inf")] * (parts - len(best))
    return sum(v >= tops[k - 1] for v in row)


def with_candidates(E, k, n, rng):
    """A row of E distinct logits of which exactly n are candidates: a part's only high value is the
    k-th largest of the maxima, and the others of the n lie in the k - 1 parts above."""
    lpt, vpl = forward(1 << 20, E, k)[:2]
    part = parts_of(lpt, vpl)[:E]
    names = sorted(set(part))
    rng.shuffle(names)
    above, last = names[:k - 1], names[k - 1]
    row = [-10.0 - 0.01 * c for c in range(E)]
    at = [c for c in range(E) if part[c] in above]
    rng.shuffle(at)
    high = [next(c for c in at if part[c] == p) for p in above]
    high += [c for c in at if c not in high][:n - 1 - len(high)]
    assert len(high) == n - 1
    values = [5.0 + 0.0625 * i for i in range(n - 1)]
    rng.shuffle(values)
    for c, v in zip(high, values):
        row[c] = v
    row[rng.choice([c for c in range(E) if part[c] == last])] = 4.0
    return row


SIZES_BY_RANK = [(64, 8), (128, 8), (128, 6), (256, 8), (384, 8), (512, 7), (1000, 8), (1024, 12)]


def test_rows_with_a_number_of_candidates():
    rng = random.Random(2)
    for E, k in SIZES_BY_RANK:
        lpt, vpl, _, one, rank = forward(1 << 20, E, k)
        assert rank and not one
        for n in range(k, 41 if E > 64 else 29):
            assert candidates(with_candidates(E, k, n, rng), lpt, vpl, k) == n
