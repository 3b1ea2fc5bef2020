"""Host-only checks of the attention operators' Python side: what a call reads of its dims, which
tensors it refuses, and how its parts are built."""
import copy
import ctypes
import pickle

import pytest

from mxfp4_routed_expert_latentmoe_gb300 import attn

torch = pytest.importorskip("torch")


def _dims(**kw):
    return attn.dims(**{**dict(n_heads=8, n_kv_heads=2, head_dim=128), **kw})


def test_copies_of_dims_stand_for_themselves():
    """What a call reads is the copy's memory, not that of the original (which may be gone)."""
    d = _dims(window=7)
    for e in (copy.copy(d), copy.deepcopy(d), pickle.loads(pickle.dumps(d)), attn.Dims.from_buffer_copy(d)):
        assert e.addr == ctypes.addressof(e) != d.addr
        assert bytes(e) == bytes(d)
        e.n_heads, e.window = 16, 9
        assert (d.n_heads, d.window) == (8, 7)
        # the native side sees the copy's heads: it asks for queries of them
        with pytest.raises(ValueError, match=r"q: a CUDA tensor .1, 16, 128."):
            attn.qk_norm_rope(e, torch.zeros(1, 8, 128), *[None] * 7)
