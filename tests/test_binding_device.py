"""Every tensor of a call has to be in device memory: the binding refuses host tensors and tensors of another device,
with or without a stream given, before the library sees an address (no GPU needed: the tensors only say where they are)."""
import pytest
import torch

from bit_delta_tenant_gb300 import bitdelta as bd

BF16, F32, I32, U8, E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float8_e4m3fn


class OnDevice(torch.Tensor):
    """A host tensor that says it is on a CUDA device."""
    is_cuda = True
    index = 0

    def get_device(self):
        return self.index


class OnAnother(OnDevice):
    index = 1


class Library:
    """Stands for the library: records whether a call got that far."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    recorder = Library()
    monkeypatch.setattr(bd, "_lib", recorder)
    return recorder


def t(*shape, dtype=BF16):
    return torch.empty(shape, dtype=torch.uint8 if dtype is E4M3 else dtype).view(dtype).as_subclass(OnDevice)


def kv(e4m3):
    pool, scale = (3, 2, 16, 64), (3, 2, 16)
    return dict(k=t(*pool, dtype=E4M3 if e4m3 else BF16), v=t(*pool, dtype=E4M3 if e4m3 else BF16),
                **(dict(k_scale=t(*scale, dtype=U8), v_scale=t(*scale, dtype=U8)) if e4m3 else {}))


def step_calls():
    cache = bd.KVCache(**kv(False))
    i = lambda *s: t(*s, dtype=I32)  # noqa: E731
    f = lambda *s: t(*s, dtype=F32)  # noqa: E731
    return [
        (bd.bd_rmsnorm, dict(x=t(4, 256), weight=t(3, 256), y=t(4, 256), residual=t(4, 256), residual_out=t(4, 256),
                             weight_ids=i(4)), dict(eps=1e-5)),
        (bd.bd_rmsnorm, dict(x=t(4, 256), weight=t(256), y=t(4, 256, dtype=E4M3), y_scale=f(4, 2)), dict(eps=1e-5)),
        (bd.bd_kv_append, dict(q=t(5, 4, 64), k=t(5, 2, 64), v=t(5, 2, 64), positions=i(5), page_table=i(2, 3), rope=f(48, 64),
                               q_out=t(5, 4, 64), seq_ids=i(5)), dict(cache=cache)),
        (bd.bd_kv_read, dict(page_table=i(2, 3), offsets=i(3), k_out=t(7, 2, 64), v_out=t(7, 2, 64)), dict(cache=cache)),
        (bd.bd_attention_decode, dict(q=t(2, 4, 64), page_table=i(2, 3), lengths=i(2), out=t(2, 4, 64),
                                      workspace=t(4096, dtype=U8), lse=f(2, 4)), dict(cache=cache)),
        (bd.bd_sample, dict(logits=t(3, 100), noise=f(3, 100), ids=i(3), temperature=f(3), top_k=i(3), top_p=f(3), min_p=f(3),
                            logprob=f(3)), {}),
    ]


@pytest.mark.parametrize("number", range(6))
def test_step_calls(lib, number):
    call, tensors, plain = step_calls()[number]
    call(**tensors, **plain, stream=5)
    assert lib.calls == 1
    for name, x in tensors.items():
        for other, word in ((x.as_subclass(torch.Tensor), "CUDA device"), (x.as_subclass(OnAnother), "device")):
            with pytest.raises(ValueError, match=word):
                call(**{**tensors, name: other}, **plain, stream=5)
    assert lib.calls == 1


@pytest.mark.parametrize("e4m3", [False, True])
def test_cache(lib, e4m3):
    d = kv(e4m3)
    bd.KVCache(**d)
    for name, x in d.items():
        with pytest.raises(ValueError, match="CUDA device"):
            bd.KVCache(**{**d, name: x.as_subclass(torch.Tensor)})


def test_workspace_is_contiguous(lib):
    call, tensors, plain = step_calls()[4]
    with pytest.raises(ValueError, match="contiguous"):
        call(**{**tensors, "workspace": t(8192, dtype=U8)[::2]}, **plain, stream=5)
    assert lib.calls == 0


def test_linears_and_compression(lib):
    x, w, bits, alpha, y, ws = t(4, 64), t(16, 64), t(16, 8, dtype=U8), t(1, dtype=F32), t(4, 16), t(4096, dtype=U8)
    ids = t(4, dtype=I32)
    calls = [
        lambda x, w, bits, alpha, y, ws, ids: bd.bd_linear(x, w, bits, alpha, 0, y, stream=5),
        lambda x, w, bits, alpha, y, ws, ids: bd.bd_linear_grouped(x, ids, w, [bits, bits], [alpha, alpha], [0, 0], y, ws, stream=5),
        lambda x, w, bits, alpha, y, ws, ids: bd.bd_linear_batch(bd.linear_descs([(x, w, bits, alpha, 0, y)]), ws, stream=5),
        lambda x, w, bits, alpha, y, ws, ids: bd.bd_compress(w, w, 0, bits, alpha, ws, stream=5),
        lambda x, w, bits, alpha, y, ws, ids: bd.bd_reconstruct(w, bits, alpha, 0, w, stream=5),
    ]
    used = ["x w bits alpha y", "x ids w bits alpha y ws", "x w bits alpha y ws", "w bits alpha ws", "w bits alpha"]
    given = dict(x=x, w=w, bits=bits, alpha=alpha, y=y, ws=ws, ids=ids)
    for call, names in zip(calls, used):
        before = lib.calls
        call(**given)
        assert lib.calls > before
        before = lib.calls
        for name in names.split():
            with pytest.raises(ValueError, match="CUDA device"):
                call(**{**given, name: given[name].as_subclass(torch.Tensor)})
        assert lib.calls == before
