"""CPU checks that the calls over a cache in 8 bits and dspark_tree_verify look at the device of every tensor that they are given: stand-ins
for tensors of two devices get as far as the library, which is replaced by one that only counts its calls."""
import pytest
import torch

import dspark_draft_selection_gb300 as ds

R, T, H, D, PAGE, V = 3, 2, 2, 64, 16, 9


class Elsewhere(torch.Tensor):
    """A host tensor that says it is of device 0, or of the one set."""
    at = 0
    is_cuda = True

    def get_device(self):
        return self.at


def _tensor(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Elsewhere)


def _arguments():
    cache = tuple(t.as_subclass(Elsewhere) for t in ds.q8_cache(8, PAGE, H, D, device="cpu"))
    f, rows = torch.float32, (R, T, H, D)
    common = dict(cache=cache, page_table=_tensor(R, 4), status=_tensor(1))
    return {
        "dspark_rope_append_q8": dict(common, q=_tensor(*rows, dtype=f), k=_tensor(*rows, dtype=f), v=_tensor(*rows, dtype=f), pos=_tensor(R, T),
                                      cos_sin=_tensor(4, D, dtype=f), ctx_len=_tensor(R), axis=_tensor(D // 2), n_nodes=_tensor(R),
                                      out=_tensor(*rows, dtype=f)),
        "dspark_tree_attention_q8": dict(common, q=_tensor(*rows, dtype=f), ctx_len=_tensor(R), mask=_tensor(R, T, 1), n_nodes=_tensor(R),
                                         out=_tensor(*rows, dtype=f), lse=_tensor(R, T, H, dtype=f), ws=_tensor(1024, dtype=torch.uint8)),
        "dspark_cache_commit_q8": dict(common, ctx_len=_tensor(R), path=_tensor(R, T), n_accepted=_tensor(R), out=_tensor(R)),
        "dspark_cache_read_q8": dict(common, n=_tensor(R), start=_tensor(R), out=tuple(_tensor(*rows, dtype=f) for _ in range(2))),
        "dspark_tree_verify": dict(p=_tensor(R, T, V, dtype=f), q=_tensor(R, T, V, dtype=f), tokens=_tensor(R, T), parent=_tensor(R, T),
                                   u_accept=_tensor(R, T, dtype=torch.float64), u_draw=_tensor(R, dtype=torch.float64), n_nodes=_tensor(R),
                                   out=(_tensor(R, T), _tensor(R), _tensor(R, T)), status=_tensor(1)),
    }


class _Library:
    calls = 0

    def __getattr__(self, name):
        def call(*_):
            self.calls += 1
            return 0
        return call


@pytest.fixture()
def library(monkeypatch):
    lib = _Library()
    monkeypatch.setattr(ds._binding, "lib", lambda: lib)
    monkeypatch.setattr(ds._binding, "_raw_stream", lambda _: 0)
    monkeypatch.setattr(ds._binding, "_device", lambda: 0)
    monkeypatch.setattr(ds._binding, "_devices", None, raising=False)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    return lib


@pytest.mark.parametrize("name", sorted(_arguments()))
def test_every_tensor_of_another_device_is_refused(name, library):
    given = _arguments()[name]
    getattr(ds, name)(**given)
    assert library.calls == 1
    for key, value in given.items():
        for t in value if isinstance(value, tuple) else (value,):
            t.at = 1
            with pytest.raises(ValueError, match="current device"):
                getattr(ds, name)(**given)
            t.at = 0
    assert library.calls == 1
    getattr(ds, name)(**given)
    assert library.calls == 2


@pytest.mark.parametrize("name", sorted(_arguments()))
def test_every_tensor_of_the_host_is_refused(name, library):
    given = _arguments()[name]
    for key, value in given.items():
        for i, t in enumerate(value if isinstance(value, tuple) else (value,)):
            plain = t.as_subclass(torch.Tensor)
            other = value[:i] + (plain,) + value[i + 1:] if isinstance(value, tuple) else plain
            with pytest.raises(ValueError, match="device tensors"):
                getattr(ds, name)(**dict(given, **{key: other}))
    assert library.calls == 0


def test_without_torchs_own_function_for_the_current_device(library, monkeypatch):
    monkeypatch.setattr(ds._binding, "_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    given = _arguments()["dspark_cache_commit_q8"]
    with pytest.raises(ValueError, match="current device"):
        ds.dspark_cache_commit_q8(**given)
    for value in given.values():
        for t in value if isinstance(value, tuple) else (value,):
            t.at = 1
    ds.dspark_cache_commit_q8(**given)
    assert library.calls == 1
