"""What the Python binding itself decides, without a GPU: the stream of a call that
names none, and how long arguments live."""
import types

import pytest
import torch


@pytest.fixture
def pa(monkeypatch):
    import paged_quantized_kv_gqa_gb300 as m
    monkeypatch.setattr(m, "_current_raw_stream", None)   # as in a process that has made no call yet
    return m


def with_cuda(monkeypatch, stream):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 1000 + dev, raising=False)


def test_the_current_stream_is_looked_up_at_every_call(pa, monkeypatch):
    with_cuda(monkeypatch, lambda: types.SimpleNamespace(cuda_stream=7))
    assert pa._stream(None) == 1003
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 5)
    pa._current_raw_stream = None
    assert pa._stream(None) == 1005
    assert pa._stream(42) == 42 and pa._stream(types.SimpleNamespace(cuda_stream=9)) == 9


def test_an_error_of_the_lookup_is_raised_and_not_kept(pa, monkeypatch):
    """A failed lookup must not turn into the legacy default stream, now or later."""
    def fails():
        raise RuntimeError("out of memory")
    with_cuda(monkeypatch, fails)
    with pytest.raises(RuntimeError):
        pa._stream(None)
    with_cuda(monkeypatch, lambda: types.SimpleNamespace(cuda_stream=7))
    assert pa._stream(None) == 1003


def test_no_device_yet_is_not_kept(pa, monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)
    assert pa._stream(None) is None
    with_cuda(monkeypatch, lambda: types.SimpleNamespace(cuda_stream=7))
    assert pa._stream(None) == 1003


def test_arguments_keep_their_tensors_alive():
    """pa_args holds addresses: a tensor that nothing else holds must not be freed under it."""
    import gc
    import weakref
    import paged_quantized_kv_gqa_gb300 as m
    names = ("q", "cache_k", "cache_v", "k_scale", "v_scale", "block_table", "out", "lse", "seq_lens", "seq_lens_kv",
             "cu_seqlens_q", "attn_mask", "shift_bias", "smooth_weight")
    tensors = {n: torch.zeros(4) for n in names}
    refs = [weakref.ref(t) for t in tensors.values()]
    args = m.make_args(**tensors)
    assert [getattr(args, n) for n in names] == [t.data_ptr() for t in tensors.values()]
    del tensors
    gc.collect()
    assert all(r() is not None for r in refs)
    del args
    gc.collect()
    assert all(r() is None for r in refs)
    raw = dict(q=256, cache_k=256, cache_v=256, k_scale=256, v_scale=256, block_table=256, out=256)
    assert m.make_args(**raw, lse=None).q == 256
