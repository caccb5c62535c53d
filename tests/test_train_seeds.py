"""The training example's update: the dense tensors and each table round with
random words of their own.  No GPU: the calls are recorded, not run."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

import hashed_gram_embedding_ngram_amd as ng  # noqa: E402
from tests import ref8  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_each_table_has_its_own_words(monkeypatch):
    spec = importlib.util.spec_from_file_location("train_projected_fp8", os.path.join(ROOT, "examples", "train_projected_fp8.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    used = []
    monkeypatch.setattr(ng, "ngram_adamw", lambda tensors, **kw: used.append((kw["seed"], kw["step"])))
    monkeypatch.setattr(ng, "ngram_adamw_rows", lambda *a, **kw: used.append((kw["seed"], kw["step"])))
    monkeypatch.setattr(ng, "ngram_quant_fp8", lambda *a, **kw: (None, None))
    layer = ex.Layer.__new__(ex.Layer)
    layer.dense, layer.P = None, None
    layer.table, layer.e1 = ex.Rows.__new__(ex.Rows), ex.Rows.__new__(ex.Rows)
    for t in (layer.table, layer.e1):
        t.p = t.m = t.v = t.m_scale = t.v_scale = None
    layer.sparse = ((None, None, None), (None, None, None))
    for seed in (0, 1, 2, 7):
        layer.update(5, seed=seed)
    assert len(used) == 12 and len(set(used)) == 12
    # and the words of the first elements differ
    words = [tuple(ref8.random_words(s, t, range(8))) for s, t in used]
    assert len(set(words)) == 12
