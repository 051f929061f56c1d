"""The `stream` argument: what a call allocates belongs to the stream that its kernels run
on.  Run without a GPU: the library, the streams and the devices are stand-ins, and every
tensor that a call makes is recorded with the stream that was current."""

import contextlib
import types

import pytest
import torch
from torch.overrides import TorchFunctionMode

from bit_nf4_quantized_27_b200 import binding as bd

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
FACTORIES = (torch.empty, torch.zeros, torch.Tensor.new_empty, torch.Tensor.new_zeros)


class Library:
    def __getattr__(self, name):
        return lambda *args: 512 if "bytes" in name else 0


class Recorder(TorchFunctionMode):
    def __init__(self):
        super().__init__()
        self.current, self.made = 0, []

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, self.current if s is None else s.cuda_stream
        yield
        self.current = before

    def __torch_function__(self, func, types_, args=(), kwargs=None):
        kwargs = dict(kwargs or {})
        if func in FACTORIES:
            self.made.append(self.current)
            if str(kwargs.get("device", "cpu")).startswith("cuda"):
                kwargs["device"] = "cpu"
            if kwargs.get("dtype") == U8 and len(args) == 1:  # at an address as the device's allocator gives
                raw = func(args[0] + 256, **kwargs)
                return raw[-raw.data_ptr() % 256:][:args[0]]
        return func(*args, **kwargs)


def _z(*shape, dt=BF):
    return torch.zeros(*shape, dtype=dt)


def _calls():
    M, N, K, r, n = 4, 16, 64, 8, 2
    q = types.SimpleNamespace(rows=N, cols=K, codes=_z(N, 32, dt=U8), c_struct=lambda: bd.NF4TensorC())
    pool = bd.AdapterPool(_z(n, r, K), _z(n, N, r), _z(n, dt=F32))
    groups = (_z(M, dt=I32), _z(n + 1, dt=I32))
    X, dY, A, B = _z(M, K), _z(M, N), _z(r, K), _z(N, r)
    keep = _z(M, K // 8, dt=U8)
    tensors = types.SimpleNamespace(table=_z(16, dt=U8), _ref=None)
    return {
        "dequantize": lambda s: bd.dequantize(q, stream=s),
        "linear_fwd": lambda s: bd.linear_fwd(q, A, B, 1.0, X, stream=s),
        "linear_bwd": lambda s: bd.linear_bwd(q, A, B, 1.0, X, dY, stream=s),
        "merge": lambda s: bd.merge(q, A, B, 1.0, stream=s),
        "linear_fwd_multi": lambda s: bd.linear_fwd_multi(q, [(A, B, 1.0)], [0] * M, X, stream=s),
        "linear_fwd_dropout": lambda s: bd.linear_fwd_dropout(q, A, B, 1.0, X, keep, 0.1, stream=s),
        "linear_bwd_dropout": lambda s: bd.linear_bwd_dropout(q, A, B, 1.0, X, dY, keep, 0.1, stream=s),
        "adapter_groups": lambda s: bd.adapter_groups(groups[0], n, stream=s),
        "adapters_fwd": lambda s: bd.adapters_fwd(pool, groups, X, _z(M, N), save_t=True, stream=s),
        "adapters_bwd": lambda s: bd.adapters_bwd(pool, groups, X, dY, stream=s),
        "linear_fwd_pool": lambda s: bd.linear_fwd_pool(q, pool, groups, X, stream=s),
        "linear_bwd_pool": lambda s: bd.linear_bwd_pool(q, pool, groups, X, dY, stream=s),
        "TensorList": lambda s: bd.TensorList([_z(8, dt=F32)], stream=s),
        "grad_norm": lambda s: bd.grad_norm(tensors, 1.0, stream=s),
        "grad_norm, stream by place": lambda s: bd.grad_norm(tensors, 1.0, None, None, s),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_allocations_belong_to_the_given_stream(monkeypatch, name):
    rec, given = Recorder(), types.SimpleNamespace(cuda_stream=0xabc)
    used = []
    monkeypatch.setattr(torch.cuda, "stream", rec.stream)
    monkeypatch.setattr(bd, "lib", Library)
    monkeypatch.setattr(bd, "_here", lambda *tensors: None)
    monkeypatch.setattr(bd, "_stream", lambda s=None: used.append(rec.current if s is None else s.cuda_stream))
    call = _calls()[name]
    for s, want in ((None, 0), (given, 0xabc)):
        del rec.made[:], used[:]
        with rec:
            call(s)
        ours = rec.made if name not in ("adapters_fwd", "TensorList") else rec.made[1:]  # the first is the caller's own
        assert ours and set(ours) == {want}
        assert used and set(used) == {want}
    assert rec.current == 0


def test_every_call_that_allocates_goes_by_its_stream():
    """A call with a `stream` that makes tensors runs with that stream as the current one."""
    import inspect

    seen = 0
    for f in list(vars(bd).values()) + [bd.TensorList.__init__]:
        inner = inspect.unwrap(f) if inspect.isfunction(f) else None
        if inner is None or inner.__module__ != bd.__name__ or "stream" not in inspect.signature(inner).parameters:
            continue
        text = inspect.getsource(inner)
        if any(w in text for w in ("torch.empty(", "torch.zeros(", "new_empty(", "new_workspace(", "_pool_grads(")):
            assert f is not inner, inner.__name__
            seen += 1
    assert seen >= 13
