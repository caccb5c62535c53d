"""AdamWTensors keeps the memory that its addresses name.  No GPU: only the
list is built, with stand-in checks of its tensors."""
import pytest

torch = pytest.importorskip("torch")
from torch.multiprocessing.reductions import StorageWeakRef  # noqa: E402

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402


@pytest.mark.parametrize("bits", [8, 32])
def test_a_swapped_storage_is_not_freed(bits, monkeypatch):
    """p.data = q gives the tensor other memory; the list still steps the old one, which must not be anyone else's by then."""
    monkeypatch.setattr(ng, "_arg", lambda t, *a: t.data_ptr())
    kind = torch.float32 if bits == 32 else torch.uint8
    lists = [[torch.zeros(640) for _ in range(3)], [torch.zeros(640) for _ in range(3)]]
    lists += [[torch.zeros(640, dtype=kind) for _ in range(3)] for _ in range(2)]
    lists += [[torch.zeros(5, dtype=torch.uint8) for _ in range(3)] for _ in range(2)] if bits == 8 else [None, None]
    t = ng.AdamWTensors(*lists)
    held = [x for group in lists if group for x in group]
    refs, addresses = [StorageWeakRef(x.untyped_storage()) for x in held], [x.data_ptr() for x in held]
    for x in held:
        x.data = torch.ones_like(x)
    assert not any(r.expired() for r in refs)
    named = [getattr(e, f) for f in ("p", "g", "m", "v") for e in t.c]
    assert named == addresses[:12]
    del t
    assert all(r.expired() for r in refs)
