"""Host-side refusals of the trainable block's operators: bad configurations and NULL arguments
are turned away before any device work."""
import ctypes
import types

import pytest
import torch

import self_referential_nested_b200 as S


@pytest.fixture(scope="module")
def lib():
    from self_referential_nested_b200 import build
    build.build()
    return S.load_library()


@pytest.mark.parametrize("bad,status", [
    (dict(dim=0), S.SRNL_E_INVAL),
    (dict(dim=-3), S.SRNL_E_INVAL),
    (dict(dim=8193), S.SRNL_E_UNSUPPORTED),
    (dict(eps=0.0), S.SRNL_E_INVAL),
    (dict(eps=float("inf")), S.SRNL_E_INVAL),
    (dict(eps=float("nan")), S.SRNL_E_INVAL),
    (dict(act_dtype=5), S.SRNL_E_INVAL),
])
def test_ln_create_rejects_bad_config_before_cuda(lib, bad, status):
    with pytest.raises(S.SrnlError) as e:
        S.srnl_ln_create(dict(dict(dim=64, eps=1e-6, act_dtype="f32"), **bad))
    assert e.value.status == status and lib.srnl_ln_last_error(None)


def test_ln_null_arguments_fail_cleanly(lib):
    h = ctypes.c_void_p()
    assert lib.srnl_ln_create(None, None) == S.SRNL_E_INVAL
    assert lib.srnl_ln_create(ctypes.byref(h), None) == S.SRNL_E_INVAL and h.value is None
    assert lib.srnl_ln_forward(*[None] * 7, 1, None) == S.SRNL_E_INVAL
    assert lib.srnl_ln_backward(*[None] * 10, 1, None) == S.SRNL_E_INVAL
    lib.srnl_ln_destroy(None)


@pytest.mark.parametrize("bad,status", [
    (dict(dim=0), S.SRNL_E_INVAL),
    (dict(hidden=-8), S.SRNL_E_INVAL),
    (dict(max_rows=0), S.SRNL_E_INVAL),
    (dict(activation=2), S.SRNL_E_INVAL),
    (dict(act_dtype="f32"), S.SRNL_E_UNSUPPORTED),
    (dict(dim=60), S.SRNL_E_UNSUPPORTED),
    (dict(hidden=12), S.SRNL_E_UNSUPPORTED),
    (dict(dim=65544), S.SRNL_E_UNSUPPORTED),
    (dict(max_rows=(1 << 24) + 1), S.SRNL_E_UNSUPPORTED),
])
def test_ffn_create_rejects_bad_config_before_cuda(lib, bad, status):
    with pytest.raises(S.SrnlError) as e:
        S.srnl_ffn_create(dict(dict(dim=64, hidden=128, max_rows=4), **bad))
    assert e.value.status == status and lib.srnl_ffn_last_error(None)


def test_ffn_null_arguments_fail_cleanly(lib):
    h = ctypes.c_void_p()
    assert lib.srnl_ffn_create(None, None) == S.SRNL_E_INVAL
    assert lib.srnl_ffn_create(ctypes.byref(h), None) == S.SRNL_E_INVAL and h.value is None
    assert lib.srnl_ffn_forward(*[None] * 7, 1, None) == S.SRNL_E_INVAL
    assert lib.srnl_ffn_backward(*[None] * 8, 1, None) == S.SRNL_E_INVAL
    assert lib.srnl_ffn_device_status(None) == S.SRNL_E_INVAL
    lib.srnl_ffn_destroy(None)


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), S.SRNL_E_INVAL),
    (dict(T=-1), S.SRNL_E_INVAL),
    (dict(heads=0), S.SRNL_E_INVAL),
    (dict(d=48), S.SRNL_E_UNSUPPORTED),
    (dict(d=256), S.SRNL_E_UNSUPPORTED),
    (dict(act_dtype="f32"), S.SRNL_E_UNSUPPORTED),
    (dict(B=40000), S.SRNL_E_UNSUPPORTED),
    (dict(T=(1 << 24) + 1), S.SRNL_E_UNSUPPORTED),
    (dict(ld=64), S.SRNL_E_INVAL),
    (dict(ld=132), S.SRNL_E_INVAL),
])
def test_lattn_create_rejects_bad_config_before_cuda(lib, bad, status):
    cfg = dict(dict(B=2, T=8, heads=2, d=64), **bad)
    with pytest.raises(S.SrnlError) as e:
        S.srnl_lattn_create(cfg, [0.9] * cfg["heads"])
    assert e.value.status == status and lib.srnl_lattn_last_error(None)


@pytest.mark.parametrize("decay", [[0.0, 0.5], [1.5, 0.5], [0.5, float("nan")], [-0.1, 0.5], [0.5], [0.5, 0.5, 0.5]])
def test_lattn_create_rejects_bad_decays_before_cuda(lib, decay):
    with pytest.raises(S.SrnlError) as e:
        S.srnl_lattn_create(dict(B=2, T=8, heads=2, d=64), decay)
    assert e.value.status == S.SRNL_E_INVAL


def test_lattn_null_arguments_fail_cleanly(lib):
    h = ctypes.c_void_p()
    assert lib.srnl_lattn_create(None, None, None) == S.SRNL_E_INVAL
    assert lib.srnl_lattn_create(ctypes.byref(h), None, None) == S.SRNL_E_INVAL and h.value is None
    assert lib.srnl_lattn_forward(*[None] * 9) == S.SRNL_E_INVAL
    assert lib.srnl_lattn_backward(*[None] * 13) == S.SRNL_E_INVAL
    assert lib.srnl_lattn_step(*[None] * 7) == S.SRNL_E_INVAL
    assert lib.srnl_lattn_device_status(None) == S.SRNL_E_INVAL
    lib.srnl_lattn_destroy(None)


@pytest.mark.parametrize("shape,full,lies", [
    ((5, 64), (5, 64), True), ((64, 5), (5, 64), False), ((2, 3, 64), (6, 64), True), ((2, 3, 4, 16), (6, 64), True),
    ((384,), (6, 64), True), ((1, 6, 1, 64), (6, 64), True), ((6, 64, 1), (6, 64), True), ((4, 96), (6, 64), False),
    ((3, 2, 64), (2, 3, 64), False), ((6, 64), (2, 3, 64), True), ((2, 192), (2, 3, 64), True), ((64, 2, 3), (2, 3, 64), False),
    ((2, 3, 8, 8), (2, 3, 8, 8), True), ((3, 2, 8, 8), (2, 3, 8, 8), False), ((2, 8, 3, 8), (2, 3, 8, 8), False),
    ((1, 1), (1,), True), ((), (1, 1), True), ((7,), (1,), False), ((7,), (1, 7), True), ((7, 1), (1, 7), True), ((14,), (7,), False),
])
def test_shapes_that_lie_as_they_should(shape, full, lies):
    h = types.SimpleNamespace(_device=-1)   # of a host tensor
    t = torch.zeros(shape, dtype=torch.bfloat16)
    if lies:
        assert S._dense(h, t, "call", "x", torch.bfloat16, full) == t.data_ptr()
        return
    with pytest.raises(S.SrnlError) as e:
        S._dense(h, t, "call", "x", torch.bfloat16, full)
    assert e.value.status == S.SRNL_E_INVAL and "x must be" in str(e.value)


def test_dense_tensors_of_no_rows_and_other_kinds():
    h = types.SimpleNamespace(_device=-1)
    assert S._dense(h, None, "call", "x", torch.float32, (4,)) == 0
    S._dense(h, torch.zeros(0, 40), "call", "x", torch.float32, (0, 40))
    for bad in (torch.zeros(4, dtype=torch.float64), torch.zeros(5), torch.zeros(8)[::2], torch.zeros(0)):
        with pytest.raises(S.SrnlError):
            S._dense(h, bad, "call", "x", torch.float32, (4,))
    with pytest.raises(S.SrnlError):   # on another device than the handle
        S._dense(types.SimpleNamespace(_device=0), torch.zeros(4), "call", "x", torch.float32, (4,))


def test_the_current_stream_without_private_names(monkeypatch):
    """Another torch may lack the short way to the current stream's address; the public one gives the same."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=4711))
    monkeypatch.setattr(torch, "_C", types.SimpleNamespace())
    assert S._stream(None) == 4711
    assert S._stream(12) == 12 and S._stream(types.SimpleNamespace(cuda_stream=34)) == 34
