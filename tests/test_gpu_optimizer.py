"""GPU tests of the gradient norm and of AdamW over a list of tensors.

32-bit states: the bits of adamw_step on each tensor.  8-bit states: codes and scales are
the bits of the float32 definition (every operation is rounded to nearest, and numpy
rounds the same way), over several steps so that each reads the states the last one
wrote; the parameters differ by the roundings counted there.  The norm is
summed in float64 and rounded once to float32: half a step, 2^-24, and as much again
for the sums in another order."""

import math

import numpy as np
import pytest
import torch

from bit_nf4_quantized_27_b200 import binding as bd
from oracle import many_adapters as MA

pytestmark = pytest.mark.gpu

SIZES = [1, 7, 255, 256, 257, 2048, 2049, 0, 70001, 16, 4096]
HP = dict(lr=2e-3, beta1=0.9, beta2=0.995, eps=1e-8, weight_decay=0.01)


def _draw(sizes, seed, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(z, generator=g) * std).to(dtype) for z in sizes]


def _cuda(ts):
    return [t.cuda() for t in ts]


def _unaligned(ts):
    """The same values at addresses that are aligned to their elements only."""
    out = []
    for i, t in enumerate(ts):
        buf = torch.empty(t.numel() + 16, dtype=t.dtype, device="cuda")
        v = buf[1 + i % 3:1 + i % 3 + t.numel()]
        v.copy_(t)
        out.append(v)
    return out


@pytest.mark.parametrize("sizes", [[1], [5, 2048, 3], SIZES, [3] * 500])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm(sizes, dtype):
    grads = _draw(sizes, len(sizes), 3.0, dtype)
    want = math.sqrt(sum(float((t.double() ** 2).sum()) for t in grads))
    ws = bd.new_workspace(bd.workspace_bytes_grad_norm())
    for place in (_cuda, _unaligned):
        tl = bd.TensorList(place(grads))
        for max_norm in (0.0, want / 3, 1e9, float("inf")):
            got = bd.grad_norm(tl, max_norm, ws=ws).tolist()
            assert abs(got[0] - want) <= 2.0 ** -23 * want
            assert abs(got[1] - min(1.0, max_norm / (want + 1e-6))) <= 2.0 ** -22


def test_norm_is_the_same_every_time_and_survives_extremes():
    big = _draw([100000, 3], 1, 1e25) + [torch.full((5,), 1e-30)]
    tl = bd.TensorList(_cuda(big))
    first = bd.grad_norm(tl, 1.0)
    want = math.sqrt(sum(float((t.double() ** 2).sum()) for t in big))
    assert abs(float(first[0]) - want) <= 2.0 ** -23 * want
    assert all(torch.equal(first, bd.grad_norm(tl, 1.0)) for _ in range(5))
    zero = bd.grad_norm(bd.TensorList([torch.zeros(9, device="cuda")]), 1.0)
    assert zero.tolist() == [0.0, 1.0]
    empty = bd.grad_norm(bd.TensorList([torch.zeros(0, device="cuda")]), 1.0)
    assert empty.tolist() == [0.0, 1.0]


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("bits", [8, 32])
def test_a_norm_that_is_not_finite_changes_nothing(bad, bits):
    st = _state([300, 2049], 3, bits, torch.float32)
    st["g"][1][700] = bad
    before = [t.clone() for k in st for t in st[k]]
    tl = _list(st, bits)
    clip = bd.grad_norm(tl, 1.0)
    assert not math.isfinite(float(clip[0])) and math.isnan(float(clip[1]))
    bd.adamw_multi(tl, 1, clip=clip, **HP)
    after = [t for k in st for t in st[k]]
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, after))


def _state(sizes, seed, bits, gdtype, place=_cuda):
    st = {"p": place(_draw(sizes, seed)), "p16": place(_draw(sizes, seed, 1.0, torch.bfloat16)),
          "g": place(_draw(sizes, seed + 1, 0.05, gdtype))}
    if bits == 32:
        st["m"], st["v"] = place([torch.zeros(z) for z in sizes]), place([torch.zeros(z) for z in sizes])
    else:
        codes = lambda: place([torch.zeros(z, dtype=torch.uint8) for z in sizes])  # noqa: E731
        scales = lambda: place([torch.zeros(-(-z // 256)) for z in sizes])  # noqa: E731
        st["m"], st["v"], st["ms"], st["vs"] = codes(), codes(), scales(), scales()
    return st


def _list(st, bits, lr_scale=None, p16=True):
    more = dict(exp_avg_scale=st["ms"], exp_avg_sq_scale=st["vs"]) if bits == 8 else {}
    return bd.TensorList(st["g"], st["p"], st["m"], st["v"], p_bf16=st["p16"] if p16 else None, lr_scale=lr_scale, **more)


@pytest.mark.parametrize("gdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("place", [_cuda, _unaligned])
def test_32_bit_states_are_adamw_step_on_each_tensor(gdtype, place):
    sizes = [z for z in SIZES if z]
    st = _state(SIZES, 5, 32, gdtype, place)
    one = _state(sizes, 5, 32, torch.float32)
    for k in ("p", "m", "v"):
        for a, b in zip(one[k], [t for t in st[k] if t.numel()]):
            a.copy_(b)
    tl = _list(st, 32)
    for step in (1, 2, 3):
        grads = _draw(SIZES, 40 + step, 0.05, gdtype)
        for t, g in zip(st["g"], grads):
            t.copy_(g)
        bd.adamw_multi(tl, step, **HP)
        for i, g in enumerate(g for g in grads if g.numel()):
            bd.adamw_step(one["p"][i], g.float().cuda(), one["m"][i], one["v"][i], step, p_bf16=one["p16"][i], **HP)
    for k in ("p", "m", "v", "p16"):
        for a, b in zip(one[k], [t for t in st[k] if t.numel()]):
            assert torch.equal(a, b), k


def test_learning_rate_scales_and_clipping():
    st = _state([300, 2049], 6, 32, torch.float32)
    ref = {k: [t.clone() for t in st[k]] for k in st}
    clip = torch.tensor([4.0, 0.25], device="cuda")
    bd.adamw_multi(_list(st, 32, lr_scale=[1.0, 16.0], p16=False), 2, clip=clip, **HP)
    for i, s in enumerate((1.0, 16.0)):
        hp = {**HP, "lr": HP["lr"] * s}
        bd.adamw_step(ref["p"][i], ref["g"][i] * 0.25, ref["m"][i], ref["v"][i], 2, **hp)
        # lr is rounded to float32 before the scale, or after it: the update differs by 2^-24 of itself, the result by a rounding
        assert torch.equal(st["m"][i], ref["m"][i]) and torch.equal(st["v"][i], ref["v"][i])
        assert ((st["p"][i] - ref["p"][i]).abs() <= 2.0 ** -22 * (ref["p"][i].abs() + s)).all()
    assert all(torch.equal(a, b) for a, b in zip(st["p16"], ref["p16"]))  # no copy asked for: not touched


@pytest.mark.parametrize("gdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("place", [_cuda, _unaligned])
def test_8_bit_states_are_the_definition(gdtype, place):
    sizes = [1, 7, 255, 256, 257, 2049, 0, 5000, 16]
    st = _state(sizes, 7, 8, gdtype, place)
    lr_scale = [1.0 + i for i in range(len(sizes))]
    tl = _list(st, 8, lr_scale)
    ref = [dict(p=t.cpu().numpy().copy(), m=np.zeros(z, np.float32), v=np.zeros(z, np.float32),
                ms=np.zeros(-(-z // 256), np.float32), vs=np.zeros(-(-z // 256), np.float32)) for t, z in zip(st["p"], sizes)]
    clip = torch.tensor([2.0, 0.75], device="cuda")
    for step in (1, 2, 3):
        grads = _draw(sizes, 60 + step, 0.05, gdtype)
        grads[5][:256] = 0.0  # a block of zeros
        grads[5][256:400] *= 1e-6  # far below its block's largest
        grads[7][0] = 300.0  # one element above all others of its block
        for t, g in zip(st["g"], grads):
            t.copy_(g)
        bd.adamw_multi(tl, step, clip=clip, seed=90 + step, **HP)
        for i, s in enumerate(ref):
            if sizes[i]:
                before = s["p"] * (1 - HP["lr"] * lr_scale[i] * HP["weight_decay"])
                s["p"], s["m"], s["v"], s["ms"], s["vs"] = MA.adamw8(
                    s["p"], grads[i].float().numpy(), s["m"], s["v"], s["ms"], s["vs"], step, i, 90 + step, clip=0.75,
                    lr_scale=lr_scale[i], **HP)
                s["update"] = before - s["p"]
            else:
                s["update"] = s["p"]
        for i, s in enumerate(ref):
            m = st["m"][i].cpu().view(torch.float8_e4m3fn).float().numpy()
            v = st["v"][i].cpu().view(torch.float8_e5m2).float().numpy()
            assert np.array_equal(st["ms"][i].cpu().numpy(), s["ms"]) and np.array_equal(st["vs"][i].cpu().numpy(), s["vs"])
            assert np.array_equal(m, s["m"]) and np.array_equal(v, s["v"]), (step, i)
            # the update's root, its scaling, the sum with eps, the product and the quotient are each off by at most two
            # steps of 2^-23 in the kernel and half a step in the definition, the result by half a step in each: 2^-19 of
            # the update and 2^-23 of the parameter, in every step taken so far
            off = np.abs(st["p"][i].cpu().numpy().astype(np.float64) - s["p"])
            s["off"] = s.get("off", 0) + 2.0 ** -19 * np.abs(s["update"]) + 2.0 ** -23 * np.abs(s["p"])
            assert np.all(off <= s["off"]), (step, i)
            assert torch.equal(st["p16"][i], st["p"][i].to(torch.bfloat16))


def test_stochastic_rounding_is_unbiased():
    """The variance of a constant gradient: each element is rounded up or down to an E5M2 value, up
    with the probability of its place between them.  n elements' mean is within 6 standard
    deviations (at most half a step over sqrt(n)) of the value; rounding to nearest would be off by up to
    half a step itself."""
    n = 1 << 18
    g = torch.full((n,), 0.83)
    g[::256] = 1.0  # sets each block's scale
    st = _state([n], 8, 8, torch.float32)
    st["g"][0].copy_(g)
    bd.adamw_multi(_list(st, 8), 1, seed=5, **HP)
    v = st["v"][0].view(torch.float8_e5m2).float().view(-1, 256)[:, 1:] / 57344.0
    m = st["m"][0].view(torch.float8_e4m3fn).float().view(-1, 256)[:, 1:] / 448.0
    assert abs(float(v.double().mean()) - 0.83 ** 2) < 6 * 0.0625 / math.sqrt(v.numel())
    assert abs(float(m.double().mean()) - 0.83) < 6 * 0.03125 / math.sqrt(m.numel())
    assert v.unique().numel() == 2 and m.unique().numel() == 2
    other = _state([n], 8, 8, torch.float32)
    other["g"][0].copy_(g)
    bd.adamw_multi(_list(other, 8), 1, seed=6, **HP)
    assert not torch.equal(other["v"][0], st["v"][0])


def test_a_small_variance_is_not_rounded_to_zero():
    g = torch.full((256,), 1e-7)
    g[0] = 1.0
    st = _state([256], 9, 8, torch.float32)
    st["g"][0].copy_(g)
    bd.adamw_multi(_list(st, 8), 1, **HP)
    assert (st["v"][0] > 0).all()


def test_a_variance_follows_its_gradients_over_many_steps():
    """With default arguments each step rounds by other random bits.  The first step's gradients are
    0.9 of their block's largest, the others' 0.3 of it; the 8-bit variance has to follow.  A rounding is off
    by less than a step of E5M2, at most 1/7 of the block's largest value, with a standard deviation of at most half
    of it; 200 of them, and n independent elements, leave the mean within 6 sqrt(200) / 14 / sqrt(n) of the exact recursion."""
    n, steps = 1 << 18, 200
    st = _state([n], 10, 8, torch.float32)
    tl = _list(st, 8, p16=False)
    exact = top = 0.0
    for step in range(1, steps + 1):
        g = 0.9 if step == 1 else 0.3
        st["g"][0].fill_(g)
        st["g"][0][::256] = 1.0
        bd.adamw_multi(tl, step, **HP)
        exact, top = HP["beta2"] * exact + (1 - HP["beta2"]) * g * g, HP["beta2"] * top + (1 - HP["beta2"])
    v = st["v"][0].view(torch.float8_e5m2).double().view(-1, 256)[:, 1:] * st["vs"][0].double()[:, None]
    assert abs(float(st["vs"][0].double().mean()) * 57344 / top - 1) < 1e-4
    assert abs(float(v.mean()) - exact) / top < 6 * math.sqrt(steps) / 14 / math.sqrt(v.numel())
