"""Host-side refusals of the paged cache's entry points for prompts and shared pages (CPU only: every
call here returns before any CUDA call)."""

import ctypes

import pytest
import torch

from tests.test_paged_abi import BAD_PAGED, GOOD, INVALID, UNSUPPORTED, WORKSPACE
from token_sparse_attention_gb300 import build as mcs_build
from token_sparse_attention_gb300 import mcs

BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    mcs_build.build()
    return mcs.lib()


def _good(p):
    """Arguments that pass the checks: (name, function, arguments, indices of required pointers)."""
    r = ctypes.byref(p)
    return [
        ("attn", "mcs_paged_attn", [r, 3, 16, 16, 16, 16, 16, 16, 16, None, 16, BIG, None], (2, 3, 4, 5, 6, 7, 8)),
        ("shared", "mcs_paged_decode_shared", [r, 2, 16, 16, 16, 16, 16, 16, 16, 16, None, 16, BIG, None], (2, 3, 4, 5, 6, 7, 8, 9)),
        ("fork", "mcs_paged_fork", [r, 3, 16, 16, 16, 16, 16, 4, 16, 32, 32, 16, 16, 16, 16, 16, BIG, None],
         (2, 3, 4, 5, 6, 8, 9, 10, 11, 12, 13, 14)),
        ("compact", "mcs_paged_compact", [r, 16, 16, 16, 16, 16, 16, 4, 16, 16, 3, 16, BIG, None], (1, 2, 3, 4, 5, 6, 8, 9)),
        ("copy", "mcs_paged_copy", [r, 3, 16, 16, 16, None, None], (2, 3, 4))]


@pytest.mark.parametrize("change,status", BAD_PAGED, ids=lambda x: str(x))
def test_params_are_checked(L, change, status):
    p = mcs.paged(**{**GOOD, **change})
    for name, f, args, _ in _good(p):
        assert getattr(L, f)(*args) == status, name
    for f in (mcs.mcs_paged_attn_workspace, mcs.mcs_paged_decode_shared_workspace, mcs.mcs_paged_fork_workspace,
              mcs.mcs_paged_compact_workspace):
        assert f(p) == 0


def test_pointers_are_checked(L):
    p = mcs.paged(**GOOD)
    for name, f, args, pointers in _good(p):
        call = getattr(L, f)
        assert call(None, *args[1:]) == INVALID
        for i in pointers:
            for bad in (None, 18):
                assert call(*args[:i], bad, *args[i + 1:]) == INVALID, (name, i, bad)
        if name in ("attn", "shared"):  # lse
            assert call(*args[:-4], 18, *args[-3:]) == INVALID
        if name != "copy":
            need = getattr(mcs, f + "_workspace")(p)
            assert need > 0
            for ws, size in ((None, BIG), (16, need - 1), (8, BIG)):
                assert call(*args[:-3], ws, size, None) == WORKSPACE, name
    assert L.mcs_paged_copy(ctypes.byref(p), 3, 16, 16, 16, 24, None) == INVALID


def test_sizes_are_checked(L):
    p = mcs.paged(**GOOD)
    attn, shared, fork, compact, copy = ((getattr(L, f), args) for _, f, args, _ in _good(p))

    def call(which, i, value):
        f, args = which
        return f(*args[:i], value, *args[i + 1:])

    assert call(attn, 1, -1) == INVALID and call(attn, 1, (1 << 30) + 1) == UNSUPPORTED
    assert call(attn, 1, 1 << 29) == UNSUPPORTED  # T * Hq
    assert attn[0](attn[1][0], 0, *[None] * 8, None, 0, None) == 0  # no rows: nothing to do
    for groups in (0, -1, GOOD["B"] + 1):
        assert call(shared, 1, groups) == INVALID
    assert call(fork, 1, 0) == INVALID and call(fork, 1, 4097) == UNSUPPORTED
    assert call(fork, 7, -1) == INVALID and call(fork, 7, (1 << 30) + 1) == UNSUPPORTED
    assert call(fork, 9, 16) == INVALID and call(fork, 10, 16) == INVALID  # lens_out, table_out are their inputs
    assert call(compact, 7, -1) == INVALID and call(compact, 7, (1 << 30) + 1) == UNSUPPORTED
    assert call(compact, 10, -1) == INVALID and call(compact, 10, (1 << 28) + 1) == UNSUPPORTED
    assert call(copy, 1, -1) == INVALID and call(copy, 1, (1 << 28) + 1) == UNSUPPORTED
    assert copy[0](copy[1][0], 0, None, None, None, None, None) == 0


def test_binding_refuses_what_does_not_fit(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    p, f = mcs.paged(**GOOD), lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)
    i = lambda *s: f(*s, t=torch.int32)
    cache, big = f(9, 2, 16, 128), lambda *s, t=torch.int32: torch.empty(*s, dtype=t, device="meta")
    with pytest.raises(ValueError, match="CUDA"):
        mcs.mcs_paged_attn(p, f(3, 8, 128), cache, cache, i(2, 4), i(2), i(3), f(3, 8, 128), f(256))
    with pytest.raises(ValueError, match="q must be"):
        mcs.mcs_paged_attn(p, f(8, 128), cache, cache, i(2, 4), i(2), i(3), f(3, 8, 128), f(256))
    with pytest.raises(ValueError, match="q: "):
        mcs.mcs_paged_attn(p, big((1 << 32) + 3, 8, 128, t=torch.bfloat16), cache, cache, i(2, 4), i(2), i(3), f(3, 8, 128), f(256))
    with pytest.raises(ValueError, match="CUDA"):
        mcs.mcs_paged_decode_shared(p, f(2, 8, 128), cache, cache, i(2, 4), i(2), i(2), i(1), f(2, 8, 128), f(256))
    with pytest.raises(ValueError, match="shared_pages must be"):
        mcs.mcs_paged_decode_shared(p, f(2, 8, 128), cache, cache, i(2, 4), i(2), i(2), i(1, 1), f(2, 8, 128), f(256))
    with pytest.raises(ValueError, match="CUDA"):
        mcs.mcs_paged_fork(p, i(3), i(2), i(2, 4), i(9), i(4), i(1), i(3), i(3, 4), i(9), i(4), i(1), i(3, 3), f(256))
    with pytest.raises(ValueError, match="parents"):
        mcs.mcs_paged_fork(p, big(1 << 32), i(2), i(2, 4), i(9), i(4), i(1), i(3), i(3, 4), i(9), i(4), i(1), i(3, 3), f(256))
    with pytest.raises(ValueError, match="free_pages"):
        mcs.mcs_paged_fork(p, i(3), i(2), i(2, 4), i(9), big(1 << 32), i(1), i(3), i(3, 4), i(9), i(4), i(1), i(3, 3), f(256))
    with pytest.raises(ValueError, match="CUDA"):
        mcs.mcs_paged_compact(p, i(2), i(2, 4), i(9), i(2, 4), i(9), i(4), i(1), i(3, 3), f(256))
    with pytest.raises(ValueError, match="moves must be"):
        mcs.mcs_paged_compact(p, i(2), i(2, 4), i(9), i(2, 4), i(9), i(4), i(1), i(9), f(256))
    with pytest.raises(ValueError, match="moves"):
        mcs.mcs_paged_copy(p, big(1 << 32, 3), cache, cache)
    with pytest.raises(ValueError, match="CUDA"):
        mcs.mcs_paged_copy(p, i(3, 3), cache, cache)
