"""Host-side checks (CPU) of the expert layer's entry points at their edges."""

import ctypes
import os

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from moe_token_block_amd import build as b
    if not os.path.exists(b.LIB):
        b.build()
    import moe_token_block_amd as m
    return m.lib()


@pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake pointers: only where no GPU exists")
def test_matvec_of_an_empty_batch_with_the_null_ids_of_an_empty_tensor(lib):
    P, N = ctypes.c_void_p(0x1000), None         # never dereferenced: every call below does nothing or is refused
    mv = lib.ep_nvfp4_expert_matvec
    for swiglu in (0, 1):
        for per_entry in (0, 1):
            for idx in (0, 1):
                assert mv(N, 0, 64, per_entry, P, 8, 16, N, idx, 2, swiglu, N, N, N) == 0
    assert mv(N, 0, 64, 0, P, 1, 16, N, 0, 1, 0, N, N, N) == 0           # dense
    # what is refused for any number of tokens still is, and NULL ids still mean one dense matrix otherwise
    assert mv(N, 0, 100, 0, P, 8, 16, N, 0, 2, 0, N, N, N) == -2
    assert mv(N, 0, 64, 0, P, 1025, 16, N, 0, 2, 0, N, N, N) == -2
    assert mv(N, 0, 64, 0, P, 8, 15, N, 0, 2, 1, N, N, N) == -2
    assert mv(N, 0, 64, 0, P, 8, 16, N, 3, 2, 0, N, N, N) == -5
    assert mv(N, 0, 64, 0, P, 8, 16, N, 0, 1025, 0, N, N, N) == -8
    assert mv(P, 1, 64, 0, P, 8, 16, N, 0, 2, 0, P, N, N) == -2


@pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake pointers: only where no GPU exists")
def test_combine_by_ids_refuses_what_its_header_excludes(lib):
    P, N = ctypes.c_void_p(0x1000), None
    c = lib.ep_bf16_combine_topk
    assert c(P, 8, 0, 4, 2, P, P, 0, 4, P, P, N) == -2
    assert c(P, 8, 8, 4, 0, P, P, 0, 4, P, P, N) == -2
    assert c(P, 8, 8, 4, 2, P, P, 0, 0, P, P, N) == -2           # no experts
    assert c(P, 8, 8, 4, 2, P, P, 0, 1025, P, P, N) == -2
    assert c(P, 8, 8, 4, 2, P, P, 2, 4, P, P, N) == -5           # index dtype
    assert c(P, 8, 8, 4, 1025, P, P, 0, 4, P, P, N) == -8
    assert c(P, 1 << 25, 8, 4, 2, P, P, 0, 4, P, P, N) == -8
    assert c(P, 8, 8, 4, 2, P, N, 0, 4, P, P, N) == -1
    assert c(P, 8, 8, 4, 2, N, P, 0, 4, P, P, N) == -1
    assert c(N, 8, 8, 4, 2, P, P, 0, 4, P, P, N) == -1
    assert c(P, 8, 8, 4, 2, P, P, 0, 4, P, N, N) == -1
    assert c(N, 0, 8, 0, 2, N, N, 1, 4, N, N, N) == 0
    for big in ((1 << 63) - 1, -(1 << 63), -1, 1 << 62, 1 << 32):
        assert c(P, big, 8, 4, 2, P, P, 0, 4, P, P, N) < 0
        assert c(P, 8, big, 4, 2, P, P, 0, 4, P, P, N) < 0
        assert c(P, 8, 8, big, 2, P, P, 0, 4, P, P, N) < 0
        assert c(P, 8, 8, 4, big, P, P, 0, 4, P, P, N) < 0
        assert c(P, 8, 8, 4, 2, P, P, 0, big, P, P, N) < 0
