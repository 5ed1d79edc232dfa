"""Paged cache kernels on the GPU: calls at the edges of what the documentation allows."""
import threading

import numpy as np
import pytest
import torch

import oracle
from kv_cache_attention_chunk_b200 import build, vkv
from test_gpu_paged import DEV, TYPES, attn_call, attn_case, attn_ref, bits, check_attn, f64, i32, new_err

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    vkv.lib()


def test_attn_refuses_an_empty_selection():
    """A selection of no entries has no address: it must not be taken for no selection."""
    c = attn_case(R=2, H=4, Hkv=2, d=64, P=16, lens=[40, 5], poison=False)
    for sel in (torch.empty((2, 2, 0), dtype=torch.int32, device=DEV), i32(np.zeros((2, 2, 3)).tolist())[:, :, :0]):
        for window in (0, 7):
            with pytest.raises(ValueError, match="sel"):
                attn_call({**c, "sel": sel, "window": window})
