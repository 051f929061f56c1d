"""What the autograd wrapper of the pool layer asks the library for.  Run without a GPU: the
calls are recorded and answered by stand-ins."""

import types

import pytest
import torch

from bit_nf4_quantized_27_b200 import binding as bd

M, N, K, R, S = 5, 16, 64, 8, 2
Q = types.SimpleNamespace(rows=N, cols=K)


def _z(*shape, dt=torch.bfloat16):
    return torch.zeros(*shape, dtype=dt)


@pytest.fixture
def calls(monkeypatch):
    made = []

    def fwd(q, pool, groups, X, save_t=True, ws=None, **kw):
        made.append(("fwd", save_t, ws))
        return _z(M, N), _z(3, M, R) if save_t else None

    def bwd(q, pool, groups, X, dY, T=None, ws=None, need_grads=True, **kw):
        made.append(("layer", need_grads, T is not None, ws))
        return (_z(M, K) + 1, *((_z(S, R, K) + 2, _z(S, N, R) + 3) if need_grads else (None, None)))

    def grads(pool, groups, X, dY, T=None, dX=None, need_grads=True, grad_dtype=torch.float32, ws=None, **kw):
        assert dX is None and grad_dtype == torch.bfloat16
        made.append(("adapters", need_grads, T is not None, ws))
        return _z(S, R, K) + 2, _z(S, N, R) + 3

    monkeypatch.setattr(bd, "linear_fwd_pool", fwd)
    monkeypatch.setattr(bd, "linear_bwd_pool", bwd)
    monkeypatch.setattr(bd, "adapters_bwd", grads)
    return made


def _run(need, *more):
    X, A, B = (t.requires_grad_(n) for t, n in zip((_z(M, K), _z(S, R, K), _z(S, N, R)), need))
    groups = _z(M, dt=torch.int32), _z(S + 1, dt=torch.int32)
    Y = bd.QLoRAPoolLinearFunction.apply(X, A, B, Q, groups, _z(S, dt=torch.float32), *more)
    if any(need):
        Y.sum().backward()
    return X.grad, A.grad, B.grad


@pytest.mark.parametrize("need", [(x, a, b) for x in (False, True) for a in (False, True) for b in (False, True)])
def test_only_the_gradients_that_are_required_are_computed(calls, need):
    x, a, b = need
    got = _run(need)
    want = [("fwd", a or b, None)]
    if x:
        want.append(("layer", a or b, a or b, None))
    elif a or b:
        want.append(("adapters", True, True, None))
    assert calls == want
    for g, n, value in zip(got, need, (1, 2, 3)):
        assert (g is not None and bool((g == value).all())) if n else g is None


@pytest.mark.parametrize("need_x", [False, True])
def test_both_directions_use_the_callers_workspace(calls, need_x):
    ws = _z(256, dt=torch.uint8)
    _run((need_x, True, True), None, ws)
    assert len(calls) == 2 and all(c[-1] is ws for c in calls)


@pytest.mark.parametrize("layer", ["one adapter", "pool"])
def test_a_second_derivative_is_refused(calls, monkeypatch, layer):
    """The gradients come from kernels that autograd does not see: differentiating them would
    leave out everything behind them."""
    X = _z(M, K).requires_grad_()
    if layer == "pool":
        groups = _z(M, dt=torch.int32), _z(S + 1, dt=torch.int32)
        Y = bd.QLoRAPoolLinearFunction.apply(X, _z(S, R, K), _z(S, N, R), Q, groups, _z(S, dt=torch.float32))
    else:
        monkeypatch.setattr(bd, "linear_fwd", lambda *a: (_z(M, N), _z(2, M, R)))
        monkeypatch.setattr(bd, "linear_bwd", lambda *a: (_z(M, K) + 1, _z(R, K), _z(N, R)))
        Y = bd.QLoRALinearFunction.apply(X, _z(R, K), _z(N, R), Q, 1.0)
    dX, = torch.autograd.grad((Y * Y).sum(), X, create_graph=True)
    with pytest.raises(RuntimeError):
        (dX * X).sum().backward()


class _Library:
    def __getattr__(self, name):
        return lambda *args: 512 if "bytes" in name else 0


@pytest.fixture
def library(monkeypatch):
    monkeypatch.setattr(bd, "lib", _Library)
    monkeypatch.setattr(bd, "_here", lambda *tensors: None)
    monkeypatch.setattr(bd, "_stream", lambda stream=None: 0)


def test_calls_tell_autograd_what_they_wrote(library):
    """Each tensor of the caller's that a call writes gets a new version, and no other does."""
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    pool = bd.AdapterPool(_z(S, R, K), _z(S, N, R), _z(S, dt=f32))
    q = types.SimpleNamespace(rows=N, cols=K, codes=_z(N, 32, dt=u8), c_struct=lambda: bd.NF4TensorC())
    idx, groups, ws = _z(M, dt=i32), (_z(M, dt=i32), _z(S + 1, dt=i32)), _z(1 << 16, dt=u8)
    X, Y, dY, dX, T = _z(M, K), _z(M, N), _z(M, N), _z(M, K), _z(3, M, R)
    outs = _z(S, R, K), _z(S, N, R)
    p, flat, g, m, v = (_z(40, dt=f32) for _ in range(5))
    p16, clip = _z(40), _z(2, dt=f32)
    tl = bd.TensorList([g, g[:8]], [p, flat[8:16]], [m, m[:8]], [v, v[:8]], p_bf16=[p16, p16[:8]])
    read = [idx, X, dY, pool.A, pool.B, pool.scales, g]
    for call, wrote in [
            (lambda: bd.adapter_groups(idx, S, out=groups, ws=ws), groups),
            (lambda: bd.adapters_fwd(pool, groups, X, Y, t_out=T, ws=ws), (Y, T)),
            (lambda: bd.adapters_bwd(pool, groups, X, dY, T, dX=dX, outs=outs, ws=ws), (dX, *outs)),
            (lambda: bd.linear_fwd_pool(q, pool, groups, X, out=Y, t_out=T, ws=ws), (Y, T)),
            (lambda: bd.linear_bwd_pool(q, pool, groups, X, dY, T, outs=(dX, *outs), ws=ws), (dX, *outs)),
            (lambda: bd.linear_bwd_pool(q, pool, groups, X, dY, T, outs=(dX, None, None), need_grads=False, ws=ws), (dX,)),
            (lambda: bd.grad_norm(tl, 1.0, out=clip, ws=ws), (clip,)),
            (lambda: bd.adamw_multi(tl, 1, 1e-3, clip=clip), (p, flat, p16))]:
        every = [*read, *groups, Y, dX, T, *outs, p, flat, p16, clip]
        before = [t._version for t in every]
        call()
        for t, b in zip(every, before):
            assert (t._version > b) == any(t is w for w in wrote)


def test_groups_written_again_before_the_backward_are_noticed(calls, library):
    """The backward would take the gradients by the new batch's groups."""
    idx, groups = _z(M, dt=torch.int32), (_z(M, dt=torch.int32), _z(S + 1, dt=torch.int32))
    X = _z(M, K).requires_grad_()
    Y = bd.QLoRAPoolLinearFunction.apply(X, _z(S, R, K), _z(S, N, R), Q, groups, _z(S, dt=torch.float32))
    bd.adapter_groups(idx, S, out=groups, ws=_z(256, dt=torch.uint8))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        Y.sum().backward()


@pytest.mark.parametrize("layer", ["one adapter", "pool"])
def test_the_backward_gets_contiguous_rows(monkeypatch, layer):
    """The kernels read X's rows one behind the other: a transposed or expanded input is copied for
    both directions, or the backward would read other rows, or past the last."""
    seen = []
    note = lambda X, out: (seen.append((X.is_contiguous(), X.clone())), out)[1]  # noqa: E731
    x = torch.arange(M * K, dtype=torch.float32).view(K, M).to(torch.bfloat16)
    X = x.clone().requires_grad_()
    if layer == "pool":
        monkeypatch.setattr(bd, "linear_fwd_pool", lambda q, p, g, X, **kw: note(X, (_z(M, N), _z(3, M, R))))
        monkeypatch.setattr(bd, "linear_bwd_pool", lambda q, p, g, X, *a, **kw: note(X, (_z(M, K), _z(S, R, K), _z(S, N, R))))
        groups = _z(M, dt=torch.int32), _z(S + 1, dt=torch.int32)
        Y = bd.QLoRAPoolLinearFunction.apply(X.t(), _z(S, R, K), _z(S, N, R), Q, groups, _z(S, dt=torch.float32))
    else:
        monkeypatch.setattr(bd, "linear_fwd", lambda q, A, B, alpha, X: note(X, (_z(M, N), _z(2, M, R))))
        monkeypatch.setattr(bd, "linear_bwd", lambda q, A, B, alpha, X, *a: note(X, (_z(M, K), _z(R, K), _z(N, R))))
        Y = bd.QLoRALinearFunction.apply(X.t(), _z(R, K), _z(N, R), Q, 1.0)
    Y.sum().backward()
    assert len(seen) == 2 and all(c and torch.equal(v, x.t()) for c, v in seen)


def test_the_layers_calls_refuse_strided_rows(library):
    q = types.SimpleNamespace(rows=N, cols=K, c_struct=lambda: bd.NF4TensorC())
    ws = _z(1 << 16, dt=torch.uint8)
    A, B, dY, keep = _z(R, K), _z(N, R), _z(M, N), _z(M, K // 8, dt=torch.uint8)
    calls = [lambda X: bd.linear_bwd(q, A, B, 1.0, X, dY, ws=ws),
             lambda X: bd.linear_fwd_multi(q, [(A, B, 1.0)], [0] * M, X, ws=ws),
             lambda X: bd.linear_fwd_dropout(q, A, B, 1.0, X, keep, 0.1, ws=ws),
             lambda X: bd.linear_bwd_dropout(q, A, B, 1.0, X, dY, keep, 0.1, ws=ws)]
    for call in calls:
        call(_z(M, K))
        for X in (_z(K, M).t(), _z(1, K).expand(M, K), _z(M, K, dt=torch.float32), _z(M, 2 * K)[:, :K]):
            with pytest.raises(AssertionError):
                call(X)
    with pytest.raises(AssertionError):
        bd.linear_bwd_dropout(q, A, B, 1.0, _z(M, K), _z(N, M).t(), keep, 0.1, ws=ws)
