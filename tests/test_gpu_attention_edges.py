"""attention_paged where its definition ends: rows that see nothing in tiles of their own, scores and weights at the
ends of their ranges, workspaces that hold anything, captured calls whose keys are dealt out anew at each replay.
Bounds as in test_gpu_attention.py unless stated."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import Setup, dev, w4  # noqa: E402, F401


@pytest.mark.parametrize("page", [16, 64, 12])
@pytest.mark.parametrize("hq,hkv,d,e4m3", [(2, 1, 64, False), (4, 2, 64, True), (16, 2, 128, False), (2, 1, 128, True),
                                           (2, 1, 256, False), (16, 2, 256, True), (4, 2, 96, False)])
def test_row_tiles_that_see_no_key(w4, hq, hkv, d, e4m3, page):  # noqa: F811
    # more new tokens than cached ones, so that the first tiles of 64 or 128 rows see nothing; no cached tokens at all;
    # alone, beside others, with tables that are split in parts
    for lens, window in (([(200, 0)], 0), ([(300, 20)], 0), ([(300, 1)], 5), ([(150, 60), (150, 2000), (90, 0)], 0),
                         ([(1, 5), (260, 0), (2, 0), (140, 200), (130, 7)], 33), ([(700, 0), (650, 700)], 0)):
        s = Setup(lens, hq, hkv, d, page, e4m3, seed=d + page)
        print(lens, window, flush=True)
        s.check(s.run(w4, window=window), window=window)
