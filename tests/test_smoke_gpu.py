"""The smoke run reaches every operator of the library (needs a B200)."""
import pytest

import __graft_entry__ as entry
from top_sparse_attention_02_b200 import binding as tsa

pytestmark = pytest.mark.gpu


def test_smoke_reaches_the_step_and_the_paged_path(cuda_dev, monkeypatch):
    called = set()
    for name in ("decode_step", "block_summarize", "qk_norm_rope", "paged_append", "paged_attn", "prefix_attn"):
        def call(*a, _f=getattr(tsa, name), _name=name, **kw):
            called.add(_name)
            return _f(*a, **kw)

        monkeypatch.setattr(tsa, name, call)
    before = tsa.launch_count()
    entry.smoke()
    assert called == {"decode_step", "block_summarize", "qk_norm_rope", "paged_append", "paged_attn", "prefix_attn"}
    assert tsa.launch_count() - before >= 18
