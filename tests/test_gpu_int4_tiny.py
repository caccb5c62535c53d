"""The 4-bit product of x near fp32's smallest numbers, in every product kernel.

Tolerance: test_gpu_int4's, and what the three bf16 parts of an fp32 x leave: bits below bf16's smallest
number, 2^-133, less than that for each x, times 31 scale (16 + q, where the group's sum of x keeps them).
Sums and factors below 2^-126 round to steps of 2^-149: one more for each addition of a group and each group."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests import ref_vocab as ref  # noqa: E402
from tests.ref_vocab import U  # noqa: E402
from tests.test_gpu_int4 import matrix  # noqa: E402
from tests.test_gpu_norm8 import BF, F32, dev  # noqa: E402
from tests.test_gpu_parity import say  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,k,o", [(3, 264, 40), (40, 264, 40), (20, 264, 33000), (70, 264, 33000)])
def test_tiny_x(n, k, o, dtype):
    say(f"4-bit tiny {n} x {k} x {o} {dtype}")
    rng, group = np.random.default_rng(n + o), 64
    w, values, scales = matrix(rng, o, k, group, True, F32)
    for e in (-100, -109, -112, -118, -124, -127):
        x = dev(((rng.random((n, k)) + 1) * 2.0 ** e * rng.choice([-1, 1], (n, k))).astype(np.float32), dtype)
        xv = x.double().cpu().numpy()
        want, groups = xv @ values.T, scales.shape[1]
        size = np.stack([np.abs(xv[:, g * group:(g + 1) * group]).sum(axis=1) for g in range(groups)], axis=1)
        bound = 1.01 * (156 * (group + 1) * U * (size @ scales.T) + 2 * (groups + 10) * U * (np.abs(xv) @ np.abs(values).T))
        most = scales.sum(axis=1)[None]
        bound = bound + (31 * group * 2.0 ** -133 * most if dtype == F32 else 0) + 2.0 ** -149 * (2 * group * most + 2 * groups)
        for ydtype in (F32, BF):
            got = ng.ngram_project_int4(x, w, dtype=ydtype).double().cpu().numpy()
            lim = bound + ref.half_step(np.abs(want) + bound, ydtype == BF)
            err = np.abs(got - want)
            assert np.all(err <= lim), (e, (err / lim).max())
