"""The random words of tables: equal places round alike under one seed and step,
and apart under two."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests.test_gpu_norm8 import BF, DEV, dev  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu


def test_seeds_of_tables():
    say("seeds of two tables")
    rng = np.random.default_rng(1)
    R, d = 64, 264
    p0, g = rng.normal(size=(R, d)) * 0.02, dev(rng.normal(size=(R, d)) * 1e-3, BF)
    rows = torch.arange(R, dtype=torch.int32, device=DEV)

    def step(seed):
        p = dev(p0, BF)
        m, v = (torch.zeros((R, d), dtype=torch.uint8, device=DEV) for _ in range(2))
        ms, vs = (torch.full((R, 3), 127, dtype=torch.uint8, device=DEV) for _ in range(2))
        ng.ngram_adamw_rows(p, m, v, rows, g, m_scale=ms, v_scale=vs, lr=1e-5, step=1, seed=seed)
        return p.view(torch.int16), m, v

    one, same, other = step(3), step(3), step(4)
    for a, b, c in zip(one, same, other):
        assert torch.equal(a, b)
        # a value between two neighbours goes up in one of the two and down in the other with a chance of up to a half
        assert 0.1 < float((a != c).float().mean()) < 0.6
