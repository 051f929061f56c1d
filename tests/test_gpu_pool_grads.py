"""GPU tests of the pool's gradients where their kernels differ: groups split over the CTAs
of a cluster, T summed beside U, and groups so long that an accumulator's chain of
additions has to be cut.  Bounds as in test_gpu_pool."""

import pytest
import torch

from bit_nf4_quantized_27_b200 import binding as bd
from test_gpu_pool import _check_all, _pool, _setup

pytestmark = pytest.mark.gpu

# m, n_out, k, r, n, lengths of the adapters' groups (None: random), ranks (None: all r).  Each has few units and
# at least 1024 tokens an adapter, so the split kernel takes it (test_pool_rules_cpu.py holds these to its rule).
SPLIT = [
    (1024, 264, 200, 24, 1, [1024], None),
    (2500, 264, 200, 24, 1, [2499], None),  # an odd tail, and one token without an adapter
    (8192, 136, 328, 64, 1, None, None),
    (3100, 264, 200, 24, 3, [2900, 0, 137], None),  # unequal groups, one of them empty
    (3333, 136, 200, 72, 3, [1, 17, 3300], None),
    (3200, 200, 264, 64, 3, None, [24, 64, 8]),
    (3200, 200, 264, 200, 3, None, [136, 200, 0]),
    (2050, 8, 8, 8, 2, None, None),
]
# The same sums over so many tokens that accumulators start anew several times, by each of the two kernels.
LONG = [(32768, 264, 200, 24, 1, True), (32768, 264, 200, 24, 40, False), (131072, 136, 72, 64, 1, True),
        (100003, 136, 72, 72, 128, False)]


def _given(m, lengths):
    if lengths is None:
        return None
    idx = torch.cat([torch.full((c,), a, dtype=torch.int32) for a, c in enumerate(lengths)])
    idx = torch.cat([idx, torch.full((m - len(idx),), -1, dtype=torch.int32)])
    return idx[torch.randperm(m, generator=torch.Generator().manual_seed(m))]


@pytest.mark.parametrize("case", SPLIT, ids=lambda c: "x".join(map(str, c[:5])))
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("saved", [True, False])
def test_groups_split_over_ctas(case, dt, saved):
    m, n_out, k, r, n, lengths, ranks = case
    _check_all(m, n_out, k, r, n, 200, dt, ranks=ranks, junk=ranks is not None, saved=saved, given=_given(m, lengths))


def test_groups_split_back_to_back():
    """Calls without a pause, whose inputs are written right ahead of each: the same bits as
    one at a time, and the same every time."""
    m, n_out, k, r, n = 2500, 264, 200, 24, 2
    sets = []
    for i in range(5):
        idx, A, B, scales, X, dY = _setup(m, n_out, k, r, n, 220 + i)
        sets.append((bd.adapter_groups(idx.cuda(), n), _pool(A, B, scales, None), X.cuda(), dY.cuda()))
    ws = bd.new_workspace(bd.workspace_bytes_adapters(m, n_out, k, r, True))
    here = [torch.empty_like(t) for t in sets[0][2:]]

    def step(groups, pool, X, dY):
        for t, new in zip(here, (X, dY)):
            t.copy_(new)
        dX = torch.zeros(m, k, device="cuda")
        return dX, *bd.adapters_bwd(pool, groups, *here, dX=dX, ws=ws)

    alone = []
    for s in sets:
        alone.append(step(*s))
        torch.cuda.synchronize()
    for _ in range(4):
        got = [step(*s) for s in sets]
        assert all(torch.equal(x, y) for a, g in zip(alone, got) for x, y in zip(a, g))
    assert bd.read_status(ws) == 0


@pytest.mark.parametrize("m,n_out,k,r,n,ranks", [
    (1, 64, 64, 8, 1, None), (300, 520, 576, 64, 5, None), (257, 384, 320, 128, 3, None), (129, 128, 1032, 200, 2, None),
    (190, 328, 264, 64, 5, [8, 64, 24, 0, 56]), (190, 328, 264, 256, 5, [200, 136, 0, 256, 40]), (9000, 264, 328, 64, 60, None)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_t_summed_beside_u(m, n_out, k, r, n, ranks, dt):
    """The backward without the forward's T: both sums in one launch."""
    _check_all(m, n_out, k, r, n, 240, dt, ranks=ranks, junk=ranks is not None, saved=False)


@pytest.mark.parametrize("case", LONG, ids=lambda c: "x".join(map(str, c[:5])))
def test_sums_over_many_tokens(case):
    """Almost all tokens in one group.  The error's root mean square stays within 2^-18 of the
    result's however many tokens there are."""
    m, n_out, k, r, n, _ = case
    g = torch.Generator(device="cuda").manual_seed(m + n)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    X, dY = normal(m, k).to(torch.bfloat16), normal(m, n_out).to(torch.bfloat16)
    A, B = (normal(n, r, k) * k ** -0.5).to(torch.bfloat16), (normal(n, n_out, r) * 0.05).to(torch.bfloat16)
    idx = torch.zeros(m, dtype=torch.int32, device="cuda")
    idx[::1000] = n - 1
    idx[5::999] = -1
    pool = bd.AdapterPool(A, B, torch.full((n,), 0.75, device="cuda"))
    ws = bd.new_workspace(bd.workspace_bytes_adapters(m, n_out, k, r, True))
    dA, dB = bd.adapters_bwd(pool, bd.adapter_groups(idx, n), X, dY, ws=ws)
    assert bd.read_status(ws) == 0
    at = (idx == 0).nonzero().view(-1)
    x, dy = X[at].double(), dY[at].double()
    U, T = dy @ B[0].double(), x @ A[0].double().t()
    for name, got, want in (("dA", dA[0], 0.75 * (U.t() @ x)), ("dB", dB[0], 0.75 * (dy.t() @ T))):
        off = float((got.double() - want).norm() / want.norm())
        assert off <= 2.0 ** -18, f"{name}: {off * 2 ** 18:.2f} of 2^-18"


@pytest.mark.parametrize("n,r,length", [(300, 8, 40008), (300, 64, 22016), (160, 136, 20008), (40, 24, 40008), (3, 200, 20008)])
def test_sums_over_a_long_dimension(n, r, length):
    """T over a long K and U over a long N: with many adapters one CTA has the whole sum, with few it is
    split.  The error's root mean square stays within 2^-18 of the result's."""
    m, short = 2 * n, 64
    g = torch.Generator(device="cuda").manual_seed(n + r)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    V, W = normal(m, length), normal(n, r, length)
    idx = torch.arange(m, dtype=torch.int32, device="cuda") % n
    groups = bd.adapter_groups(idx, n)
    ones = torch.ones(n, device="cuda")
    want = torch.stack([W[a].double() @ V[t].double() for t, a in enumerate(idx.tolist())])  # [m, r]

    def hold(name, got, ref):
        off = float((got.double() - ref).norm() / ref.norm())
        assert off <= 2.0 ** -18, f"{name}: {off * 2 ** 18:.2f} of 2^-18"

    ws = bd.new_workspace(bd.workspace_bytes_adapters(m, short, length, r, True))
    B = torch.zeros(n, short, r, dtype=torch.bfloat16, device="cuda")
    T = bd.adapters_fwd(bd.AdapterPool(W, B, ones), groups, V, torch.zeros(m, short, device="cuda"), save_t=True, ws=ws)
    hold("T", T.double().sum(0), want)
    # U = dY B with B = W^T; A has a one in each row, so dX holds U
    A = torch.zeros(n, r, 256, dtype=torch.bfloat16, device="cuda")
    A[:, torch.arange(r), torch.arange(r)] = 1.0
    pool = bd.AdapterPool(A, W.transpose(1, 2).contiguous(), ones)
    X = torch.zeros(m, 256, dtype=torch.bfloat16, device="cuda")
    for grads in (False, True):  # U alone, and beside T
        dX = torch.zeros(m, 256, device="cuda")
        bd.adapters_bwd(pool, groups, X, V, dX=dX, need_grads=grads, grad_dtype=torch.bfloat16, ws=ws)
        hold("U", dX[:, :r], want)
    assert bd.read_status(ws) == 0
