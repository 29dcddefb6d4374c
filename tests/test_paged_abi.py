"""Host-side refusals of the paged-cache and norm-with-rotation entry points (CPU only:
every call here returns before any CUDA call)."""

import ctypes

import pytest
import torch

from token_sparse_attention_gb300 import build as mcs_build
from token_sparse_attention_gb300 import mcs

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    mcs_build.build()
    return mcs.lib()


GOOD = dict(B=2, Hq=8, Hkv=2, D=128, page=16, num_pages=9, max_pages=4)

BAD_PAGED = [
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=7), INVALID), (dict(Hq=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(D=256), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
    (dict(page=256), UNSUPPORTED), (dict(B=4097), UNSUPPORTED),
    (dict(B=4096, Hq=1024), UNSUPPORTED), (dict(num_pages=1 << 27), UNSUPPORTED),
    (dict(max_pages=1 << 27), UNSUPPORTED), (dict(kv=2), INVALID), (dict(kv=-1), INVALID),
    (dict(kv=1, k_scale=0.0), INVALID), (dict(kv=1, v_scale=float("inf")), INVALID),
    (dict(kv=1, k_scale=float("nan")), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(q_stride=1016), INVALID),
    (dict(kv=1, scale=1e10, k_scale=1e30), INVALID), (dict(scale=3e38), INVALID),
    (dict(q_stride=1028), INVALID), (dict(kv_stride=248), INVALID), (dict(kv_stride=-256), INVALID),
]


def _calls(L, p):
    """Each paged entry point with pointers that pass the checks."""
    r, n = ctypes.byref(p), 1 << 40
    return {
        "plan": lambda: L.mcs_paged_plan(r, 16, 16, 16, 4, 16, 16, 16, 16, 16, 16, None, 4, None),
        "write": lambda: L.mcs_paged_write(r, 3, 16, 16, 16, 16, 16, None, None),
        "decode": lambda: L.mcs_paged_decode(r, 16, 16, 16, 16, 16, 16, None, 16, n, None),
        "select": lambda: L.mcs_paged_select(r, 16, 16, 16, 16, 2, 1, 1, 16, 16, n, None),
        "sparse": lambda: L.mcs_paged_decode_sparse(r, 16, 16, 16, 16, 16, 16, 2, 16, None, 16, n,
                                                    None),
    }


@pytest.mark.parametrize("change,status", BAD_PAGED, ids=lambda x: str(x))
def test_paged_params_are_checked(L, change, status):
    p = mcs.paged(**{**GOOD, **change})
    for name, call in _calls(L, p).items():
        assert call() == status, name
    assert mcs.mcs_paged_decode_workspace(p) == 0
    assert mcs.mcs_paged_select_workspace(p) == 0


def test_paged_struct_and_workspaces(L):
    assert ctypes.sizeof(mcs.Paged) == 13 * 4
    p = mcs.paged(**GOOD)
    assert mcs.mcs_paged_decode_workspace(p) > 0
    assert mcs.mcs_paged_select_workspace(p) >= 2 * 2 * 4 * 4
    assert L.mcs_paged_decode_workspace(None) == 0 and L.mcs_paged_select_workspace(None) == 0


def test_paged_pointers_are_checked(L):
    p = mcs.paged(**GOOD)
    r, n = ctypes.byref(p), 1 << 40
    # plan: required pointers, then sizes
    plan = [16, 16, 16, 4, 16, 16, 16, 16, 16, 16, None, 4]
    for i in (0, 1, 2, 4, 5, 6, 7, 8, 9):
        for bad in (None, 18):
            assert L.mcs_paged_plan(r, *plan[:i], bad, *plan[i + 1:], None) == INVALID, i
    assert L.mcs_paged_plan(r, *plan[:10], 18, 4, None) == INVALID
    assert L.mcs_paged_plan(r, *plan[:11], -1, None) == INVALID
    assert L.mcs_paged_plan(r, *plan[:3], -1, *plan[4:], None) == INVALID
    assert L.mcs_paged_plan(r, *plan[:11], (1 << 30) + 1, None) == UNSUPPORTED
    assert L.mcs_paged_plan(r, *plan[:3], (1 << 30) + 1, *plan[4:], None) == UNSUPPORTED
    assert L.mcs_paged_plan(None, *plan, None) == INVALID
    # write
    write = [16, 16, 16, 16, 16, None]
    for i in range(5):
        for bad in (None, 18):
            assert L.mcs_paged_write(r, 3, *write[:i], bad, *write[i + 1:], None) == INVALID, i
    assert L.mcs_paged_write(r, 3, *write[:5], 24, None) == INVALID
    assert L.mcs_paged_write(r, -1, *write, None) == INVALID
    assert L.mcs_paged_write(r, (1 << 30) + 1, *write, None) == UNSUPPORTED
    assert L.mcs_paged_write(r, 0, *[None] * 6, None) == 0  # no tokens: nothing to do
    # decode and its sparse form
    dec = [16, 16, 16, 16, 16, 16]
    for i in range(6):
        for bad in (None, 18):
            args = dec[:i] + [bad] + dec[i + 1:]
            assert L.mcs_paged_decode(r, *args, None, 16, n, None) == INVALID, i
            assert L.mcs_paged_decode_sparse(r, *args[:5], 16, 2, args[5], None, 16, n,
                                             None) == INVALID, i
    assert L.mcs_paged_decode(r, *dec, 18, 16, n, None) == INVALID
    assert L.mcs_paged_decode_sparse(r, *dec[:5], None, 2, 16, None, 16, n, None) == INVALID
    assert L.mcs_paged_decode_sparse(r, *dec[:5], 16, 0, 16, None, 16, n, None) == INVALID
    need = mcs.mcs_paged_decode_workspace(p)
    for ws, size in ((None, n), (16, need - 1), (8, n)):
        assert L.mcs_paged_decode(r, *dec, None, ws, size, None) == WORKSPACE
        assert L.mcs_paged_decode_sparse(r, *dec[:5], 16, 2, 16, None, ws, size, None) == WORKSPACE
    # select
    for select, sink, recent in ((0, 0, 0), (2, -1, 0), (2, 0, -1), (2, 2, 1), (3, 1 << 30, 1 << 30)):
        assert L.mcs_paged_select(r, 16, 16, 16, 16, select, sink, recent, 16, 16, n, None) == INVALID
    for i in range(4):
        args = [16] * i + [None] + [16] * (3 - i)
        assert L.mcs_paged_select(r, *args, 2, 1, 1, 16, 16, n, None) == INVALID
    assert L.mcs_paged_select(r, 16, 16, 16, 16, 2, 1, 1, None, 16, n, None) == INVALID
    assert L.mcs_paged_select(r, 16, 16, 16, 16, 2, 1, 1, 16, 16, 63, None) == WORKSPACE


ROPE = dict(B=2, N=5, Hq=4, Hkv=2, D=128, rot=64, table_rows=8)

BAD_ROPE = [
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=-1), INVALID),
    (dict(D=80), UNSUPPORTED), (dict(rot=8), UNSUPPORTED), (dict(rot=144), UNSUPPORTED),
    (dict(rot=-16), UNSUPPORTED), (dict(interleaved=2), INVALID), (dict(layout=2), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(q_stride=504), INVALID),
    (dict(q_stride=516), INVALID), (dict(k_stride=8), INVALID), (dict(table_rows=4), INVALID),
    (dict(table_rows=-1), INVALID), (dict(B=1 << 20, N=1 << 11), UNSUPPORTED),
    (dict(B=1 << 15, N=1 << 14), UNSUPPORTED), (dict(B=1, Hq=1 << 24), UNSUPPORTED),
    (dict(B=1, Hkv=1 << 25, D=64), UNSUPPORTED),
]


@pytest.mark.parametrize("change,status", BAD_ROPE, ids=lambda x: str(x))
def test_rope_params_are_checked(L, change, status):
    p = mcs.rope_params(**{**ROPE, **{k: v for k, v in change.items() if k != "interleaved"}})
    p.interleaved = change.get("interleaved", 0)
    r = ctypes.byref(p)
    assert L.mcs_qk_norm_rope(r, 16, 16, 16, 16, 16, 16, None, 16, 16, None) == status
    assert L.mcs_qk_norm_rope_backward(r, 16, 16, 16, 16, 16, 16, 16, 16, None, 16, 16, 16, 16, 16,
                                       1 << 40, None) == status
    if "table_rows" not in change or change["table_rows"] < 0:
        assert mcs.mcs_qk_norm_rope_backward_workspace(p) == 0


def test_rope_pointers_are_checked(L):
    p = mcs.rope_params(**ROPE)
    r = ctypes.byref(p)
    assert ctypes.sizeof(mcs.Rope) == 12 * 4
    fwd = [16, 16, 16, 16, 16, 16, None, 16, 16]
    for i, bad in [(0, None), (1, None), (4, None), (5, None), (7, None), (8, None), (0, 24),
                   (2, 18), (3, 18), (4, 20), (6, 18), (7, 24)]:
        assert L.mcs_qk_norm_rope(r, *fwd[:i], bad, *fwd[i + 1:], None) == INVALID, (i, bad)
    bwd = [16, 16, 16, 16, 16, 16, 16, 16, None, 16, 16, 16, 16]
    for i, bad in [(0, None), (1, None), (2, None), (3, None), (6, None), (7, None), (9, None),
                   (10, None), (9, 24), (11, 18), (12, 18)]:
        assert L.mcs_qk_norm_rope_backward(r, *bwd[:i], bad, *bwd[i + 1:], 16, 1 << 40,
                                           None) == INVALID, (i, bad)
    need = mcs.mcs_qk_norm_rope_backward_workspace(p)
    assert need > 0
    assert L.mcs_qk_norm_rope_backward(r, *bwd, 16, need - 1, None) == WORKSPACE
    assert L.mcs_qk_norm_rope_backward(r, *bwd, None, need, None) == WORKSPACE


def test_binding_refuses_host_tensors(monkeypatch):
    # the binding checks every tensor before the library is called
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    p, f = mcs.paged(**GOOD), lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)
    i = lambda *s: f(*s, t=torch.int32)
    cache = f(9, 2, 16, 128)
    with pytest.raises(ValueError, match="CUDA"):
        mcs.mcs_paged_decode(p, f(2, 8, 128), cache, cache, i(2, 4), i(2), f(2, 8, 128), f(256))
    with pytest.raises(ValueError, match="CUDA"):
        mcs.mcs_paged_write(p, f(3, 2, 128), f(3, 2, 128), i(3), cache, cache)
    with pytest.raises(ValueError, match="CUDA"):
        mcs.mcs_paged_plan(p, i(2), i(2), i(4), i(1), i(2, 4), i(2), i(1), i(3), i(3))
    with pytest.raises(ValueError, match="sel must be"):
        mcs.mcs_paged_select(p, f(2, 8, 128), f(9, 2, 128), i(2, 4), i(2), i(2, 4), f(256))
    # sizes that a C int cannot hold are refused, not cut
    big = lambda *s: torch.empty(*s, dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="slots"):
        mcs.mcs_paged_write(p, f(3, 2, 128), f(3, 2, 128), big((1 << 32) + 3), cache, cache)
    with pytest.raises(ValueError, match="slots"):
        mcs.mcs_paged_plan(p, i(2), i(2), i(4), i(1), i(2, 4), i(2), i(1), i(3), big((1 << 32) + 3))
    with pytest.raises(ValueError, match="free_pages"):
        mcs.mcs_paged_plan(p, i(2), i(2), big(1 << 31), i(1), i(2, 4), i(2), i(1), i(3), i(3))
    with pytest.raises(ValueError, match="sel"):
        mcs.mcs_paged_select(p, f(2, 8, 128), f(9, 2, 128), i(2, 4), i(2), big(2, 2, (1 << 32) + 2), f(256))
    with pytest.raises(ValueError, match="sink"):
        mcs.mcs_paged_select(p, f(2, 8, 128), f(9, 2, 128), i(2, 4), i(2), i(2, 2, 2), f(256), sink=1 << 32)
    r = mcs.rope_params(**ROPE)
    with pytest.raises(ValueError, match="CUDA"):
        mcs.mcs_qk_norm_rope(r, f(2, 5, 4, 128), f(2, 5, 2, 128), None, None, None, None, None,
                             f(2, 4, 5, 128), f(2, 2, 5, 128))
