"""GPU tests of the operators for many adapters on one base: grouping, forward,
backward and the NF4 layer with a pool beside it, against float64.

Bounds, for each element.  An intermediate (T = X A^T or U = dY B) is summed in
float32 over L products and kept in three bf16 planes, each off by at most 2^-8 of
what it rounds: 2^-24 |T| together (bf16 results may take the first two: 2^-16).  A
float32 sum of L products in any order is off by at most L 2^-23 of the sum of their
magnitudes (2^-24 for a rounding, twice that for an adder that cuts off).  So a
result of r (or, for dA and dB, of tokens) products of the intermediate is off by at
most (2^-24 + len 2^-23) mag1 + L 2^-23 mag2, with mag1 the sum of the magnitudes of
its products and mag2 the same with the intermediate's own sum of magnitudes, plus
the last rounding of the output: 2^-23 or 2^-8 of it.  These worst cases grow with the
length; the root mean square of the error, to which roundings add like a random walk, is
held to 2^-18 of the result's, or to a bf16 half step of it."""

import numpy as np
import pytest
import torch

import oracle as O
from bit_nf4_quantized_27_b200 import binding as bd
from bit_nf4_quantized_27_b200 import inputs as I
from oracle import many_adapters as MA

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _np(t):
    return t.detach().float().cpu().numpy()


def _index(m, n, seed, none=0.2, used=None):
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, n if used is None else used, (m,), generator=g, dtype=torch.int32)
    return torch.where(torch.rand(m, generator=g) < none, -1, idx).to(torch.int32)


def _setup(m, n_out, k, r, n, seed, ranks=None, none=0.2, used=None, junk=False):
    idx = _index(m, n, seed, none, used)
    A = I.normal((n, r, k), k ** -0.5, seed + 1)
    B = I.normal((n, n_out, r), 0.05, seed + 2)
    if junk:  # what lies past an adapter's rank is not used
        for i, rk in enumerate(ranks):
            A[i, rk:] = float("nan")
            B[i, :, rk:] = float("inf")
    scales = 0.5 + torch.rand(n, generator=torch.Generator().manual_seed(seed + 3))
    X, dY = I.normal((m, k), 1.0, seed + 4), I.normal((m, n_out), 1.0, seed + 5)
    return idx, A, B, scales, X, dY


def _pool(A, B, scales, ranks):
    return bd.AdapterPool(A.cuda(), B.cuda(), scales.cuda(), None if ranks is None else torch.tensor(ranks, dtype=torch.int32).cuda())


def _hold(name, got, ref, mag1, mag2, terms, inner, dt):
    g = _np(got).astype(np.float64)
    out = 2.0 ** -8 if dt == "bf16" else 2.0 ** -23
    bound = ((2.0 ** -16 if dt == "bf16" else 2.0 ** -24) + terms * 2.0 ** -23) * mag1 + inner * 2.0 ** -23 * mag2
    bound = bound + out * (np.abs(ref) + bound)
    err = np.abs(g - ref)
    assert np.all(np.isfinite(g)), name
    assert np.all(err <= bound), f"{name}: {np.max(err / np.maximum(bound, 1e-300)):.2f} of the bound"
    rms = float(np.sqrt(np.mean(ref ** 2))) if ref.size else 0.0
    rel = 2.0 ** -8 if dt == "bf16" else 2.0 ** -18
    assert not ref.size or float(np.sqrt(np.mean(err ** 2))) <= rel * rms, f"{name}: rms"


def _check_all(m, n_out, k, r, n, seed, dt="f32", ranks=None, none=0.2, used=None, junk=False, saved=True,
               given=None):
    idx, A, B, scales, X, dY = _setup(m, n_out, k, r, n, seed, ranks, none, used, junk)
    idx = idx if given is None else given
    Y0, dX0 = I.normal((m, n_out), 1.0, seed + 6, DT[dt]), I.normal((m, k), 1.0, seed + 7, DT[dt])
    pool = _pool(A, B, scales, ranks)
    groups = bd.adapter_groups(idx.cuda(), n)
    Y, dX = Y0.cuda(), dX0.cuda()
    ws = bd.new_workspace(bd.workspace_bytes_adapters(m, n_out, k, r, True))
    T = bd.adapters_fwd(pool, groups, X.cuda(), Y, save_t=True, ws=ws)
    dA, dB = bd.adapters_bwd(pool, groups, X.cuda(), dY.cuda(), T if saved else None, dX=dX, grad_dtype=DT[dt], ws=ws)
    torch.cuda.synchronize()
    assert bd.read_status(ws) == 0
    args = (_np(A), _np(B), scales.numpy(), idx.numpy(), _np(X))
    ry, _, m1, m2 = MA.fwd(*args, _np(Y0), ranks)
    _hold("Y", Y, ry, m1, m2, r, k, dt)
    off = idx.numpy() < 0
    assert np.array_equal(_np(Y)[off], _np(Y0)[off]) and np.array_equal(_np(dX)[off], _np(dX0)[off])
    ref = MA.bwd(*args, _np(dY), _np(dX0), ranks)
    _hold("dX", dX, ref["dX"], ref["dX1"], ref["dX2"], r, n_out, dt)
    _hold("dA", dA, ref["dA"], ref["dA1"], ref["dA2"], m, n_out, dt)
    _hold("dB", dB, ref["dB"], ref["dB1"], ref["dB2"], m, k, dt)
    # zeros for adapters without tokens and past the rank
    for a in range(n):
        rk = r if ranks is None else ranks[a]
        empty = not bool((idx == a).any())
        assert not _np(dA)[a, 0 if empty else rk:].any() and not _np(dB)[a][:, 0 if empty else rk:].any()


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("m,n,seed", [(0, 3, 1), (1, 1, 2), (31, 5, 3), (33, 1024, 4), (1000, 7, 5), (4097, 300, 6),
                                      (70001, 1024, 7), (70001, 2, 8)])
def test_groups_are_a_stable_sort(m, n, seed):
    idx = _index(m, n, seed)
    order, offsets = bd.adapter_groups(idx.cuda(), n)
    ro, rf = MA.groups(idx.numpy(), n)
    assert np.array_equal(order.cpu().numpy(), ro) and np.array_equal(offsets.cpu().numpy(), rf)


@pytest.mark.parametrize("value", [-1, 0, 2])
def test_groups_of_one_value(value):
    idx = torch.full((777,), value, dtype=torch.int32)
    order, offsets = bd.adapter_groups(idx.cuda(), 3)
    ro, rf = MA.groups(idx.numpy(), 3)
    assert np.array_equal(order.cpu().numpy(), ro) and np.array_equal(offsets.cpu().numpy(), rf)


def test_groups_reports_values_out_of_range():
    idx = torch.tensor([0, 5, -2, 1, 3, -1, 2 ** 30, -(2 ** 31)], dtype=torch.int32)
    ws = bd.new_workspace(bd.STATUS_BYTES)
    order, offsets = bd.adapter_groups(idx.cuda(), 3, ws=ws)
    assert bd.read_status(ws) == 1
    assert offsets.tolist() == [0, 1, 2, 2] and order.tolist() == [0, 3, 1, 2, 4, 5, 6, 7]


@pytest.mark.parametrize("m,n_out,k,r,n,seed", [
    (1, 64, 64, 8, 1, 10), (1, 4096, 1024, 64, 3, 11), (5, 8, 8, 8, 2, 12), (17, 136, 200, 16, 17, 13),
    (130, 264, 72, 24, 2, 14), (300, 520, 576, 64, 5, 15), (257, 384, 320, 128, 3, 16), (200, 200, 264, 256, 2, 17),
    (129, 128, 1032, 200, 2, 18), (64, 1000, 136, 72, 40, 19)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_forward_and_gradients(m, n_out, k, r, n, seed, dt):
    _check_all(m, n_out, k, r, n, seed, dt)


def test_long_sums():
    """One adapter with all tokens, and the longest contractions of a layer."""
    _check_all(600, 2048, 2752, 64, 1, 30, none=0.0)


@pytest.mark.parametrize("n_out,k,r", [(264, 136, 16), (1160, 1096, 72)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[1, 16, 15, 17, 31, 32, 33, 47, 48, 63, 64, 65, 80, 96], [300, 3, 129], [5, 5, 5, 5]])
def test_runs_of_rows(lengths, dt, n_out, k, r):
    """Requests one behind the other, adapters in turns, one without: runs of rows of every
    length, whole and cut by tiles."""
    n = 5
    given = torch.cat([torch.full((c,), (3 * i) % n if i % 6 != 4 else -1, dtype=torch.int32) for i, c in enumerate(lengths)])
    _check_all(given.numel(), n_out, k, r, n, 33, dt, given=given)


@pytest.mark.parametrize("m,n,used", [(700, 1024, None), (700, 321, 3), (3, 1024, None), (4, 2, 1)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_many_adapters_and_few_tokens(m, n, used, dt):
    _check_all(m, 72, 80, 8, n, 35, dt, used=used, none=0.0)


def test_more_tiles_than_fit_at_once():
    """Every kernel takes several rounds; long groups beside short ones."""
    g = torch.Generator().manual_seed(36)
    given = torch.where(torch.rand(9000, generator=g) < 0.3, 1, torch.randint(0, 60, (9000,), generator=g)).to(torch.int32)
    _check_all(9000, 264, 328, 64, 60, 37, "bf16", given=given)


@pytest.mark.parametrize("r,ranks", [(64, [8, 64, 24, 0, 56]), (128, [72, 128, 8, 0, 120]), (256, [200, 136, 0, 256, 40]),
                                     (24, [24, 8, 16, 0, 24])])
def test_ranks_differ_and_padding_is_junk(r, ranks):
    _check_all(190, 328, 264, r, 5, 40 + r, ranks=ranks, junk=True)


def test_recomputed_t_gives_the_same_bits():
    idx, A, B, scales, X, dY = _setup(200, 136, 328, 24, 4, 50)
    pool, groups = _pool(A, B, scales, None), bd.adapter_groups(idx.cuda(), 4)
    T = bd.adapters_fwd(pool, groups, X.cuda(), torch.zeros(200, 136, device="cuda"), save_t=True)
    a = bd.adapters_bwd(pool, groups, X.cuda(), dY.cuda(), T)
    b = bd.adapters_bwd(pool, groups, X.cuda(), dY.cuda(), None)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("used,none", [(1, 0.0), (2, 0.9), (None, 1.0)])
def test_groups_without_tokens(used, none):
    if none == 1.0:  # no token has an adapter
        idx, A, B, scales, X, dY = _setup(40, 64, 128, 16, 6, 60, none=2.0)
        pool, groups = _pool(A, B, scales, None), bd.adapter_groups(idx.cuda(), 6)
        Y = torch.randn(40, 64, device="cuda")
        Y0 = Y.clone()
        bd.adapters_fwd(pool, groups, X.cuda(), Y)
        dA, dB = bd.adapters_bwd(pool, groups, X.cuda(), dY.cuda())
        assert torch.equal(Y, Y0) and not dA.any() and not dB.any()
    else:
        _check_all(150, 192, 136, 32, 9, 61, none=none, used=used)


def test_no_tokens():
    _, A, B, scales, X, dY = _setup(0, 64, 128, 16, 3, 70)
    pool, groups = _pool(A, B, scales, None), bd.adapter_groups(torch.empty(0, dtype=torch.int32, device="cuda"), 3)
    bd.adapters_fwd(pool, groups, X.cuda(), torch.empty(0, 64, device="cuda"))
    dA, dB = bd.adapters_bwd(pool, groups, X.cuda(), dY.cuda(), dX=torch.empty(0, 128, device="cuda"))
    assert not dA.any() and not dB.any()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_column_slices_of_wider_tensors(dt):
    """X, dY, dX and Y as columns of wider rows: the bytes beside them stay."""
    m, n_out, k, r, n = 77, 104, 136, 16, 3
    idx, A, B, scales, X, dY = _setup(m, n_out, k, r, n, 80)
    pool, groups = _pool(A, B, scales, None), bd.adapter_groups(idx.cuda(), n)
    Y = torch.randn(m, n_out, device="cuda").to(DT[dt])
    dX = torch.randn(m, k, device="cuda").to(DT[dt])
    wide = {"X": torch.zeros(m, k + 24, dtype=torch.bfloat16, device="cuda"),
            "dY": torch.zeros(m, n_out + 8, dtype=torch.bfloat16, device="cuda"),
            "Y": torch.full((m, n_out + 7), 3.0, dtype=DT[dt], device="cuda"),
            "dX": torch.full((m, k + 5), 3.0, dtype=DT[dt], device="cuda")}
    vX, vdY, vY, vdX = wide["X"][:, 8:8 + k], wide["dY"][:, 8:8 + n_out], wide["Y"][:, 3:3 + n_out], wide["dX"][:, 1:1 + k]
    vX.copy_(X), vdY.copy_(dY), vY.copy_(Y), vdX.copy_(dX)
    T = bd.adapters_fwd(pool, groups, X.cuda(), Y, save_t=True)
    g0 = bd.adapters_bwd(pool, groups, X.cuda(), dY.cuda(), T, dX=dX)
    bd.adapters_fwd(pool, groups, vX, vY)
    g1 = bd.adapters_bwd(pool, groups, vX, vdY, T, dX=vdX)
    assert torch.equal(vY, Y) and torch.equal(vdX, dX) and all(torch.equal(a, b) for a, b in zip(g0, g1))
    assert (wide["Y"][:, :3] == 3).all() and (wide["Y"][:, 3 + n_out:] == 3).all()
    assert (wide["dX"][:, :1] == 3).all() and (wide["dX"][:, 1 + k:] == 3).all()


def test_rows_far_apart():
    """Row strides of 2^30 elements: offsets past 32 bits in X, dY, Y and dX."""
    m, n_out, k, r, n, ld = 3, 72, 136, 16, 2, 1 << 30
    idx, A, B, scales, X, dY = _setup(m, n_out, k, r, n, 85, none=0.0)
    pool, groups = _pool(A, B, scales, None), bd.adapter_groups(idx.cuda(), n)
    Y, dX = torch.randn(m, n_out, device="cuda"), torch.randn(m, k, device="cuda")
    far = lambda t: torch.empty_strided(t.shape, (ld, 1), dtype=t.dtype, device="cuda").copy_(t)  # noqa: E731
    fX, fdY, fY, fdX = far(X), far(dY), far(Y), far(dX)
    bd.adapters_fwd(pool, groups, X.cuda(), Y)
    g0 = bd.adapters_bwd(pool, groups, X.cuda(), dY.cuda(), dX=dX)
    bd.adapters_fwd(pool, groups, fX, fY)
    g1 = bd.adapters_bwd(pool, groups, fX, fdY, dX=fdX)
    assert torch.equal(fY, Y) and torch.equal(fdX, dX) and all(torch.equal(a, b) for a, b in zip(g0, g1))


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace and outputs, give what they give alone."""
    sets = []
    for i, (m, n_out, k, r, n) in enumerate([(700, 520, 1096, 64, 5), (333, 1160, 328, 24, 9)]):
        idx, A, B, scales, X, dY = _setup(m, n_out, k, r, n, 86 + i)
        ws = bd.new_workspace(bd.workspace_bytes_adapters(m, n_out, k, r, True))
        sets.append((_pool(A, B, scales, None), idx.cuda(), n, X.cuda(), dY.cuda(), ws))

    def step(pool, idx, n, X, dY, ws):
        groups = bd.adapter_groups(idx, n, ws=ws)
        Y = torch.zeros(X.shape[0], dY.shape[1], device="cuda")
        dX = torch.zeros(X.shape, device="cuda")
        bd.adapters_fwd(pool, groups, X, Y, ws=ws)
        return Y, dX, *bd.adapters_bwd(pool, groups, X, dY, dX=dX, ws=ws)

    alone = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(step(*s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(alone, got) for a, b in zip(x, y))
    assert all(bd.read_status(s[-1]) == 0 for s in sets)


@pytest.mark.parametrize("m,n_out,k,r,n", [(6, 1160, 520, 64, 5), (330, 520, 1096, 24, 9), (2100, 264, 328, 64, 40)])
def test_calls_back_to_back(m, n_out, k, r, n):
    """Every buffer is written anew right ahead of the calls that read it, and read right
    after, without a pause: the same bits as one batch at a time."""
    q = bd.quantize(I.normal((n_out, 64 * (k // 64)), 0.02, 9).cuda())
    kq = q.cols
    batches = []
    for i in range(6):
        idx, A, B, scales, X, dY = _setup(m, n_out, kq, r, n, 140 + i, none=0.1 * i)
        batches.append([t.cuda() for t in (idx, A, B, scales, X, dY)])
    here = [torch.empty_like(t) for t in batches[0]]
    idx, A, B, scales, X, dY = here
    pool = bd.AdapterPool(A, B, scales)
    groups = bd.adapter_groups(idx.fill_(-1), n)
    ws = bd.new_workspace(bd.workspace_bytes_adapters(m, n_out, kq, r, True))

    def step(batch):
        for t, new in zip(here, batch):
            t.copy_(new)
        bd.adapter_groups(idx, n, out=groups, ws=ws)
        Y, T = bd.linear_fwd_pool(q, pool, groups, X, ws=ws)
        Z = Y.float()
        bd.adapters_fwd(pool, groups, X, Z, ws=ws)
        one = bd.linear_bwd_pool(q, pool, groups, X, dY, T, ws=ws)
        dX = one[0].float()
        return (Y, Z, *one, dX, *bd.adapters_bwd(pool, groups, X, dY, dX=dX, ws=ws))

    alone = []
    for b in batches:
        alone.append(step(b))
        torch.cuda.synchronize()
    for _ in range(4):
        got = [step(b) for b in batches]
        assert all(torch.equal(x, y) for a, g in zip(alone, got) for x, y in zip(a, g))
    assert bd.read_status(ws) == 0


def test_parts_of_the_backward_alone():
    idx, A, B, scales, X, dY = _setup(90, 200, 136, 32, 4, 90)
    pool, groups = _pool(A, B, scales, None), bd.adapter_groups(idx.cuda(), 4)
    dX = torch.zeros(90, 136, device="cuda")
    dA, dB = bd.adapters_bwd(pool, groups, X.cuda(), dY.cuda(), dX=dX)
    dX2 = torch.zeros(90, 136, device="cuda")
    assert bd.adapters_bwd(pool, groups, X.cuda(), dY.cuda(), dX=dX2, need_grads=False) == (None, None)
    dA2, dB2 = bd.adapters_bwd(pool, groups, X.cuda(), dY.cuda())
    assert torch.equal(dX, dX2) and torch.equal(dA, dA2) and torch.equal(dB, dB2)


def test_infinities_and_nan_stay_with_their_tokens_and_adapters():
    m, n_out, k, r, n = 160, 136, 200, 24, 3
    idx, A, B, scales, X, dY = _setup(m, n_out, k, r, n, 95, none=0.1)
    bad = (idx == 1).nonzero().view(-1)[:3]
    pool, groups = _pool(A, B, scales, None), bd.adapter_groups(idx.cuda(), n)

    def run(X, dY):
        Y, dX = torch.zeros(m, n_out, device="cuda"), torch.zeros(m, k, device="cuda")
        T = bd.adapters_fwd(pool, groups, X.cuda(), Y, save_t=True)
        return Y, dX, *bd.adapters_bwd(pool, groups, X.cuda(), dY.cuda(), T, dX=dX)

    clean = run(X, dY)
    X[bad[0], 5], X[bad[1], 7], dY[bad[2], 9] = float("nan"), float("inf"), float("nan")
    none = (idx < 0).nonzero().view(-1)[0]
    X[none] = float("nan")
    dirty = run(X, dY)
    rows = torch.ones(m, dtype=torch.bool)
    rows[bad] = False
    for i in (0, 1):
        assert torch.equal(clean[i][rows.cuda()], dirty[i][rows.cuda()])
    for i in (2, 3):
        assert torch.equal(clean[i][[0, 2]], dirty[i][[0, 2]])
    assert not torch.isfinite(dirty[0][bad[0]]).any() and not torch.isfinite(dirty[2][1]).all()


def test_orders_out_of_range_are_skipped_and_reported():
    m, n_out, k, r, n = 20, 64, 72, 8, 2
    idx, A, B, scales, X, dY = _setup(m, n_out, k, r, n, 97, none=0.0)
    pool = _pool(A, B, scales, torch.tensor([8, 8]).tolist())
    order, offsets = bd.adapter_groups(idx.cuda(), n)
    order = order.clone()
    skipped = order[3].item()
    order[3] = m + 1000
    Y = torch.zeros(m, n_out, device="cuda")
    ws = bd.new_workspace(bd.workspace_bytes_adapters(m, n_out, k, r, True))
    bd.adapters_fwd(pool, (order, offsets), X.cuda(), Y, ws=ws)
    assert bd.read_status(ws) == 1
    assert not Y[skipped].any() and all(Y[t].any() for t in range(m) if t != skipped)
    bd.clear_status(ws)
    pool = _pool(A, B, scales, [12, 8])  # not a multiple of 8
    bd.adapters_fwd(pool, (order[:0].new_tensor(range(m)), offsets), X.cuda(), Y, ws=ws)
    assert bd.read_status(ws) == 1


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("m,n_out,k", [(1, 256, 512), (16, 200, 320), (48, 264, 576), (300, 520, 1088)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_nf4_layer_with_a_pool(m, n_out, k, dt):
    """The base is held to 1e-2 of the root mean square, as the layer with one adapter is
    (bf16: and one step of the output, twice for the two roundings of Y)."""
    r, n = 16, 3
    idx, A, B, scales, X, dY = _setup(m, n_out, k, r, n, 100 + m)
    w = I.normal((n_out, k), 0.02, 7)
    q = bd.quantize(w.cuda())
    wd = _np(bd.dequantize(q, torch.float32)).astype(np.float64)
    pool, groups = _pool(A, B, scales, None), bd.adapter_groups(idx.cuda(), n)
    ws = bd.new_workspace(bd.workspace_bytes_adapters(m, n_out, k, r, True))
    Y, T = bd.linear_fwd_pool(q, pool, groups, X.cuda(), y_dtype=DT[dt], ws=ws)
    dX, dA, dB = bd.linear_bwd_pool(q, pool, groups, X.cuda(), dY.cuda(), T, dx_dtype=DT[dt], grad_dtype=DT[dt], ws=ws)
    assert bd.read_status(ws) == 0
    args = (_np(A), _np(B), scales.numpy(), idx.numpy(), _np(X))
    ry = MA.fwd(*args, _np(X).astype(np.float64) @ wd.T)[0]
    ref = MA.bwd(*args, _np(dY), _np(dY).astype(np.float64) @ wd)
    for name, got, want in (("Y", Y, ry), ("dX", dX, ref["dX"]), ("dA", dA, ref["dA"]), ("dB", dB, ref["dB"])):
        err, rms = np.abs(_np(got) - want), np.sqrt(np.mean(want ** 2))
        step = 2.0 ** -7 * np.abs(want) if dt == "bf16" else 0.0
        assert np.all(err <= 1e-2 * rms + step), name


def test_nf4_layer_without_adapters_is_the_base():
    m, n_out, k = 300, 264, 320
    idx, A, B, scales, X, _ = _setup(m, n_out, k, 8, 2, 111, none=2.0)
    q = bd.quantize(I.normal((n_out, k), 0.02, 8).cuda())
    pool, groups = _pool(A, B, scales, None), bd.adapter_groups(idx.cuda(), 2)
    Y, _ = bd.linear_fwd_pool(q, pool, groups, X.cuda(), y_dtype=torch.float32)
    zero = torch.zeros(n_out, 8, dtype=torch.bfloat16, device="cuda")
    want, _ = bd.linear_fwd(q, A[0].cuda(), zero, 1.0, X.cuda(), y_dtype=torch.float32)
    assert torch.equal(Y, want)


def test_autograd_and_differences():
    """Gradients through autograd against the formula, and against central differences: the
    loss is linear in A alone and in B alone, and inputs are small multiples of powers of
    two, so a difference is exact but for the float32 sums of the loss."""
    m, n_out, k, r, n = 40, 64, 128, 8, 2
    idx, _, _, scales, _, _ = _setup(m, n_out, k, r, n, 120)
    g = torch.Generator().manual_seed(5)
    draw = lambda *s: (torch.randint(-8, 9, s, generator=g) / 16).to(torch.bfloat16)  # noqa: E731
    A, B, X, dY = draw(n, r, k), draw(n, n_out, r), draw(m, k), draw(m, n_out)
    q = bd.quantize(I.normal((n_out, k), 0.02, 9).cuda())
    groups = bd.adapter_groups(idx.cuda(), n)
    leaves = [t.cuda().requires_grad_() for t in (X, A, B)]
    Y = bd.QLoRAPoolLinearFunction.apply(*leaves, q, groups, scales.cuda(), None)
    Y.backward(dY.cuda())
    wd = _np(bd.dequantize(q, torch.float32)).astype(np.float64)
    ref = MA.bwd(_np(A), _np(B), scales.numpy(), idx.numpy(), _np(X), _np(dY), _np(dY).astype(np.float64) @ wd)
    for name, leaf in zip(("dX", "dA", "dB"), leaves):
        err, want = np.abs(_np(leaf.grad) - ref[name]), ref[name]
        assert np.all(err <= 1e-2 * np.sqrt(np.mean(want ** 2)) + 2.0 ** -7 * np.abs(want)), name

    def loss(A, B):
        Y = torch.zeros(m, n_out, device="cuda")
        bd.adapters_fwd(_pool(A, B, scales, None), groups, X.cuda(), Y)
        return float((Y.double() * dY.cuda().double()).sum())

    h = 1 / 16
    for name, t in (("dA", A), ("dB", B)):
        D = torch.where(torch.rand(t.shape, generator=g) < 0.5, -1.0, 1.0)
        plus, minus = (t.float() + h * D).to(torch.bfloat16), (t.float() - h * D).to(torch.bfloat16)
        diff = (loss(plus, B) - loss(minus, B) if name == "dA" else loss(A, plus) - loss(A, minus)) / (2 * h)
        slope = float((ref[name] * D.double().numpy()).sum())
        # each Y is off by at most 2^-24 of its magnitudes and its sums; the loss sums them against |dY| <= 1/2
        mags = MA.fwd(_np(A), _np(B), scales.numpy(), idx.numpy(), _np(X), np.zeros((m, n_out)))[3]
        assert abs(diff - slope) <= 2 * (2.0 ** -24 + (r + k) * 2.0 ** -23) * 2 * float(mags.sum()) / (2 * h)


def test_captured_step_equals_the_eager_one():
    """Grouping, forward, backward, norm and update on a side stream, captured once and
    replayed, give the eager run's bits; so does a second replay on new inputs."""
    m, n_out, k, r, n = 210, 136, 320, 16, 4
    idx, A, B, scales, X, dY = _setup(m, n_out, k, r, n, 130)
    idx2, _, _, _, X2, dY2 = _setup(m, n_out, k, r, n, 131)
    q = bd.quantize(I.normal((n_out, k), 0.02, 10).cuda())

    class Step:
        def __init__(self):
            self.idx, self.X, self.dY = idx.cuda(), X.cuda(), dY.cuda()
            self.p = [A.float().cuda(), B.float().cuda()]
            self.p16 = [A.cuda(), B.cuda()]
            self.pool = bd.AdapterPool(*self.p16, scales.cuda())
            self.groups = torch.empty(m, dtype=torch.int32, device="cuda"), torch.empty(n + 1, dtype=torch.int32, device="cuda")
            self.Y = torch.empty(m, n_out, dtype=torch.bfloat16, device="cuda")
            self.T = torch.empty(3, m, r, dtype=torch.bfloat16, device="cuda")
            self.dX = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
            self.g = [torch.empty_like(p) for p in self.p]
            self.m = [torch.zeros(p.numel(), dtype=torch.uint8, device="cuda") for p in self.p]
            self.v = [torch.zeros(p.numel(), dtype=torch.uint8, device="cuda") for p in self.p]
            sc = lambda: [torch.zeros(-(-p.numel() // 256), device="cuda") for p in self.p]  # noqa: E731
            self.ms, self.vs = sc(), sc()
            flat = lambda ts: [t.view(-1) for t in ts]  # noqa: E731
            self.list = bd.TensorList(flat(self.g), flat(self.p), self.m, self.v, flat(self.p16), self.ms, self.vs)
            self.clip = torch.empty(2, device="cuda")
            self.ws = bd.new_workspace(max(bd.workspace_bytes_adapters(m, n_out, k, r, True), bd.workspace_bytes_grad_norm()))

        def __call__(self):
            bd.adapter_groups(self.idx, n, out=self.groups, ws=self.ws)
            bd.linear_fwd_pool(q, self.pool, self.groups, self.X, out=self.Y, t_out=self.T, ws=self.ws)
            bd.linear_bwd_pool(q, self.pool, self.groups, self.X, self.dY, self.T, outs=(self.dX, *self.g), ws=self.ws)
            bd.grad_norm(self.list, 0.3, out=self.clip, ws=self.ws)
            bd.adamw_multi(self.list, 3, 1e-3, clip=self.clip, seed=11, weight_decay=0.01)

        def state(self):
            return [self.Y, self.dX, self.clip, *self.g, *self.p, *self.p16, *self.m, *self.v, *self.ms, *self.vs]

    eager, captured = Step(), Step()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        Step()()  # first calls look up addresses and attributes
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            captured()
        for inputs in ((idx, X, dY), (idx2, X2, dY2)):
            for s in (eager, captured):
                s.idx.copy_(inputs[0]), s.X.copy_(inputs[1]), s.dY.copy_(inputs[2])
            eager()
            graph.replay()
            stream.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(eager.state(), captured.state()))
            assert bd.read_status(eager.ws) == 0 and bd.read_status(captured.ws) == 0
    assert float(eager.clip[0]) > 0 and any(x.any() for x in eager.m)


def test_a_given_stream_without_a_workspace():
    """Calls that make their own scratch and outputs on a stream that is not the current one,
    while the current stream fills memory of the same sizes as fast as it can: the bits
    of calls on the current stream alone."""
    m, n_out, k, r, n = 700, 520, 1088, 64, 5
    idx, A, B, scales, X, dY = _setup(m, n_out, k, r, n, 150)
    q = bd.quantize(I.normal((n_out, k), 0.02, 11).cuda())
    pool, idx, X, dY = _pool(A, B, scales, None), idx.cuda(), X.cuda(), dY.cuda()
    Y0, dX0 = torch.zeros(m, n_out, device="cuda"), torch.zeros(m, k, device="cuda")

    def step(stream, Y, dX):
        groups = bd.adapter_groups(idx, n, stream=stream)
        T = bd.adapters_fwd(pool, groups, X, Y, save_t=True, stream=stream)
        grads = bd.adapters_bwd(pool, groups, X, dY, dX=dX, stream=stream)
        Z, T2 = bd.linear_fwd_pool(q, pool, groups, X, stream=stream)
        more = bd.linear_bwd_pool(q, pool, groups, X, dY, T2, stream=stream)
        tl = bd.TensorList([g.view(-1) for g in grads], stream=stream)
        return (*groups, Y, dX, T, *grads, Z, T2, *more, bd.grad_norm(tl, 1.0, stream=stream)), tl

    want, _ = step(None, Y0.clone(), dX0.clone())
    side = torch.cuda.Stream()
    sizes = [bd.STATUS_BYTES, bd.workspace_bytes_grad_norm(), 2 * (n + 1) * 4]
    sizes += [bd.workspace_bytes_adapters(m, n_out, k, r, b) for b in (False, True)]
    for _ in range(20):
        Y, dX = Y0.clone(), dX0.clone()
        side.wait_stream(torch.cuda.current_stream())
        got, tl = step(side, Y, dX)
        for z in sizes * 4:
            torch.empty(z, dtype=torch.uint8, device="cuda").fill_(0xff)
        torch.cuda.synchronize()
        # rows of T without an adapter are not written
        rows = (idx >= 0)
        for a, b in zip(want, got):
            same = torch.equal(a[:, rows], b[:, rows]) if a.dim() == 3 and a.shape[:2] == (3, m) else torch.equal(a, b)
            assert same


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("r", [24, 64, 136])
def test_an_infinite_intermediate_is_the_definitions(r, dt):
    """T or U of a token is infinite: its rows of Y and dX, and all that its adapter's gradients make
    of it, are infinite or NaN where the definition's are, with the same signs."""
    m, n_out, k, n = 70, 136, 200, 2
    idx, A, B, scales, X, dY = _setup(m, n_out, k, r, n, 160, none=0.0)
    t, u = (idx == 0).nonzero().view(-1)[:2].tolist()
    at_k, at_n = 5, 9
    sign = torch.where(torch.rand(r, generator=torch.Generator().manual_seed(r)) < 0.5, -1.0, 1.0).to(torch.bfloat16)
    third = n_out // 3  # sums of infinities of one sign, of the other, and of both
    B[0, :third], B[0, third : 2 * third] = B[0, :third].abs() * sign, -B[0, third : 2 * third].abs() * sign
    A[0, :, : k // 2] = A[0, :, : k // 2].abs() * sign[:, None]
    X[t, at_k], dY[u, at_n] = float("inf"), float("-inf")
    pool, groups = _pool(A, B, scales, None), bd.adapter_groups(idx.cuda(), n)
    Y, dX = torch.zeros(m, n_out, dtype=DT[dt], device="cuda"), torch.zeros(m, k, dtype=DT[dt], device="cuda")
    T = bd.adapters_fwd(pool, groups, X.cuda(), Y, save_t=True)
    dA, dB = bd.adapters_bwd(pool, groups, X.cuda(), dY.cuda(), T, dX=dX, grad_dtype=DT[dt])
    x, dy, a, b = X.double(), dY.double(), A.double(), B.double()
    s, own = scales.double(), idx == 0
    wT = torch.stack([x[i] @ a[idx[i]].t() for i in range(m)])
    wU = torch.stack([dy[i] @ b[idx[i]] for i in range(m)])
    wY = torch.stack([s[idx[i]] * (b[idx[i]] @ wT[i]) for i in range(m)])
    wX = torch.stack([s[idx[i]] * (wU[i] @ a[idx[i]]) for i in range(m)])
    wA, wB = s[0] * (wU[own].t() @ x[own]), s[0] * (dy[own].t() @ wT[own])

    def same(got, want):
        got = got.double().cpu()
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
        assert torch.equal(got[want.isinf()], want[want.isinf()])

    assert wT[t].isinf().all() and wU[u].isinf().all() and wY[t].isinf().sum() >= n_out // 4 and wX[u].isinf().any()
    same(T[0], wT), same(Y, wY), same(dX, wX)
    assert not T[1:, t].any()
    # where the infinity itself meets the other, finite intermediate, NaN may stand for it
    keep_k, keep_n = torch.arange(k) != at_k, torch.arange(n_out) != at_n
    same(dA[0][:, keep_k.cuda()], wA[:, keep_k]), same(dB[0][keep_n.cuda()], wB[keep_n])
    assert not dA[0][:, at_k].isfinite().any() and not dB[0][at_n].isfinite().any()
    assert wA[:, keep_k].isinf().any() and wB[keep_n].isinf().any()


@pytest.mark.parametrize("need", [(True, False, False), (False, True, False), (False, False, True), (True, True, False), (True, True, True)])
def test_autograd_of_some_of_the_inputs(need):
    """The gradients asked for have the bits of all of them together."""
    m, n_out, k, r, n = 150, 136, 320, 24, 3
    idx, A, B, scales, X, dY = _setup(m, n_out, k, r, n, 170)
    q = bd.quantize(I.normal((n_out, k), 0.02, 12).cuda())
    groups = bd.adapter_groups(idx.cuda(), n)
    pool = _pool(A, B, scales, None)
    Y, T = bd.linear_fwd_pool(q, pool, groups, X.cuda())
    want = bd.linear_bwd_pool(q, pool, groups, X.cuda(), dY.cuda(), T)
    leaves = [t.cuda().requires_grad_(x) for t, x in zip((X, A, B), need)]
    got = bd.QLoRAPoolLinearFunction.apply(*leaves, q, groups, scales.cuda(), None)
    assert torch.equal(got, Y)
    got.backward(dY.cuda())
    for leaf, w, x in zip(leaves, want, need):
        assert torch.equal(leaf.grad, w) if x else leaf.grad is None


def test_autograd_reports_through_the_callers_workspace():
    m, n_out, k, r, n = 40, 64, 128, 16, 2
    idx, A, B, scales, X, dY = _setup(m, n_out, k, r, n, 180, none=0.0)
    q = bd.quantize(I.normal((n_out, k), 0.02, 13).cuda())
    ws = bd.new_workspace(bd.workspace_bytes_adapters(m, n_out, k, r, True))
    order, offsets = bd.adapter_groups(idx.cuda(), n, ws=ws)
    for bad in (False, True):
        if bad:
            order = order.clone()
            order[3] = m + 7
        leaves = [t.cuda().requires_grad_() for t in (X, A, B)]
        Y = bd.QLoRAPoolLinearFunction.apply(*leaves, q, (order, offsets), scales.cuda(), None, ws)
        assert bd.read_status(ws) == (1 if bad else 0)
        bd.clear_status(ws)
        Y.backward(dY.cuda())
        assert bd.read_status(ws) == (1 if bad else 0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_one_token_in_a_tensor_of_any_width(dt):
    n_out, k, r, n = 136, 200, 24, 2
    _, A, B, scales, X, dY = _setup(1, n_out, k, r, n, 190, none=0.0)
    pool, groups = _pool(A, B, scales, None), bd.adapter_groups(torch.tensor([1], dtype=torch.int32, device="cuda"), n)
    Y, dX = torch.ones(1, n_out, dtype=DT[dt], device="cuda"), torch.ones(1, k, dtype=DT[dt], device="cuda")
    row = lambda t, pad: torch.zeros(2, t.shape[1] + pad, dtype=t.dtype, device="cuda")[:1, : t.shape[1]].copy_(t)  # noqa: E731
    vX, vdY, vY, vdX = row(X, 4), row(dY, 1), row(Y, 3), row(dX, 5)
    bd.adapters_fwd(pool, groups, X.cuda(), Y)
    want = bd.adapters_bwd(pool, groups, X.cuda(), dY.cuda(), dX=dX)
    bd.adapters_fwd(pool, groups, vX, vY)
    got = bd.adapters_bwd(pool, groups, vX, vdY, dX=vdX)
    assert torch.equal(vY, Y) and torch.equal(vdX, dX) and all(torch.equal(a, b) for a, b in zip(got, want))
