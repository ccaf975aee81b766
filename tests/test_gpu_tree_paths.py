"""attention_paged_tree where its kernels' parts, turns and words of masks meet; bounds as in test_gpu_attention.py."""

from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import attnref  # noqa: E402
from test_gpu_attention import dev, w4  # noqa: E402, F401
from test_gpu_tree_attention import Tree, words_of  # noqa: E402


@pytest.mark.parametrize("d,e4m3", [(64, False), (64, True), (128, False), (128, True), (256, False), (256, True)])
@pytest.mark.parametrize("n", [3, 12, 16])
@pytest.mark.parametrize("old", [False, True])
def test_weights_of_few_rows_keep_22_bits(w4, d, e4m3, n, old):  # noqa: F811
    # of 16 rows at most.
    # Two keys of nearly the same score count, one with v = 1 and one with v = -1; all others have scores 16 or more below
    # theirs and v = 0.  So out = (a - b) / (a + b + the rest) is small, and its own rounding with it: 2^-11 of at most 0.032.
    # A row's a and b come from one score each: q0 k0 is exact (q and k are 0 elsewhere), times scale log2 e is off by three
    # roundings of a value below 1.45, less m (11 below the largest) one of a value below 16: 1.45 * 3 * 2^-24 + 2^-21 < 2^-20 in
    # all, times ln 2 of a weight; exp2 2^-21, two f16 2^-22.  Each is below 2^-19 off, so out below 2^-19, and the sums, of
    # 300 keys at most in blocks of 16 (which but for two weights are below 2^-23 of the largest), and the division
    # 2^-21 each.  Weights of 11 bits are off by 2^-12, and out by 2^-13.
    s = Tree([(n, n + 170)], 2, 2, d, 16, e4m3, seed=d + n, kind="tree", scales=False)
    rng = np.random.default_rng(d + n)
    # where the two stand: in a tile that all rows see whole, or among the new tokens, seen by every row (of itself and its sign)
    hot = (70, 77) if old else (170 + 1, 170 + 2)
    for t in range(n):
        s.sees[t] = s.sees[t] | {1, 2}
    s.mask = dev(words_of(s.sees, s.words))
    s.q[:] = 0
    s.q[..., 0] = rng.uniform(0.5, 1.0, (n, 2))
    code = {x: int(np.flatnonzero(attnref.e4m3_values() == x)[0]) for x in (0.0, 1.0, -1.0, 0.9375, -32.0)} if e4m3 else None

    def put(c, at, x):
        c[s.table[0, at // 16], :, at % 16, 0] = code[x] if e4m3 else x

    for c in s.host:
        c[s.table[0, :-(-(n + 170) // 16)]] = code[0.0] if e4m3 else 0.0
    for j in range(n + 170):
        put(s.host[0], j, -32.0)
    put(s.host[0], hot[0], 1.0), put(s.host[0], hot[1], 0.9375)
    for i in range(d):
        for at, x in zip(hot, (1.0, -1.0)):
            s.host[1][s.table[0, at // 16], :, at % 16, i] = code[x] if e4m3 else x
    s.dev = [s._place(c, "phtd") for c in s.host]
    got = s.run(w4, scale=1.0).cpu().numpy().astype(np.float64)
    want, size, _ = s.want(1.0)
    assert np.abs(want).max() <= 0.032 and size.max() <= 1
    err = np.abs(got - want)
    assert (err <= np.abs(want) * 2.0 ** -11 + 2.0 ** -19 + 2 * 2.0 ** -21).all(), err.max()
