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
