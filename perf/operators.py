"""Measured cases of the operators for many LoRA adapters on one frozen base.

  groups   tokens sorted by adapter (stable), with the first place of each adapter
  fwd      Y[t] += s_a (X[t] A_a^T) B_a^T beside a shared projection, a the token's adapter
  bwd      its gradients: dX[t] += s_a (dY[t] B_a) A_a, dA_a and dB_a
  norm     norm of all gradients of a list of tensors, and the factor that clips it
  adamw    one AdamW step over a list of tensors, states in 32 bits or in 8

With ``own`` false, run() computes the plain form in elementary torch operations in
float32; with ``own`` true it calls the package's entry points.
"""

import math
import random

import torch

own = False

BLOCK = 256  # elements that share one float32 scale of an 8-bit state
HYPER = dict(lr=2e-4, beta1=0.9, beta2=0.995, eps=1e-8, weight_decay=0.01)
STEP = 7


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # the tokens of one decode step, each of another request
        dict(name="groups_decode", op="groups", m=64, s=32, requests=64, none=8),
        # packed prompts of many requests before a prefill
        dict(name="groups_prefill", op="groups", m=65536, s=512, requests=1500, none=10),
        # one request, one new token, q of the 7B block
        dict(name="fwd_token", op="fwd", m=1, n=4096, k=4096, r=64, s=8, requests=1, none=0, out="bf16", mixed=False),
        # a decode batch in which every request has its own adapter and ranks differ, gate/up of the 7B block
        dict(name="fwd_decode", op="fwd", m=48, n=11008, k=4096, r=64, s=48, requests=48, none=12, out="bf16", mixed=True),
        # prompts of ragged lengths packed into one batch, with decode tokens between them
        dict(name="fwd_packed", op="fwd", m=2039, n=4096, k=4096, r=64, s=16, requests=23, none=9, out="bf16", mixed=False),
        # training eight adapters on gate/up of the 65B-shaped block
        dict(name="fwd_large", op="fwd", m=4096, n=22016, k=8192, r=64, s=8, requests=8, none=0, out="f32", mixed=False),
        # training four adapters on gate/up of the 7B block
        dict(name="bwd_train", op="bwd", m=2048, n=11008, k=4096, r=64, s=4, requests=4, none=0, out="f32", mixed=False),
        # a small ragged batch on an odd layer, ranks that are not powers of two
        dict(name="bwd_odd", op="bwd", m=1003, n=1000, k=576, r=24, s=6, requests=13, none=7, out="bf16", mixed=True),
        # the gradients of one small layer's adapters
        dict(name="norm_small", op="norm", n=1024, k=576, r=8, layers=3, grad="f32"),
        # the gradients of 32 blocks of the 7B shape at rank 8: 448 tensors
        dict(name="norm_many", op="norm", n=11008, k=4096, r=8, layers=224, grad="bf16"),
        # the adapters of one 65B-shaped block, states in 32 bits
        dict(name="adamw_32bit", op="adamw", n=22016, k=8192, r=64, layers=7, grad="f32", bits=32),
        # the adapters of 32 blocks of the 7B shape at rank 16, states in 8 bits
        dict(name="adamw_8bit", op="adamw", n=11008, k=4096, r=16, layers=224, grad="bf16", bits=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["groups", "fwd", "fwd", "bwd", "bwd", "norm", "adamw", "adamw"])
    if op == "groups":
        m = _log(rng, 16, 65536)
        return dict(op=op, m=m, s=_log(rng, 6, 1024), requests=_log(rng, 8, m), none=rng.choice([0, 3, 10]))
    if op in ("fwd", "bwd"):
        m = _log(rng, 1, 4096 if op == "fwd" else 2048)
        k, n = 64 * _log(rng, 1, 128), 8 * _log(rng, 16, 1376)
        if op == "bwd":
            n = min(n, 8192)
            k = min(k, 8192)
        r = rng.choice([8, 16, 24, 32, 64, 64, 72, 128, 256])
        s = _log(rng, 1, 64)
        while s * r * (n + k) > 64 * 64 * 15104:
            s = max(1, s // 2)
        return dict(op=op, m=m, n=n, k=k, r=r, s=s, requests=_log(rng, 1, min(m, 64)), none=rng.choice([0, 4, 9]),
                    out=rng.choice(["bf16", "f32"]), mixed=rng.random() < 0.4)
    layers = _log(rng, 1, 224)
    r = 8 * rng.randint(1, 8)
    n, k = 8 * _log(rng, 16, 1376), 64 * _log(rng, 1, 128)
    while layers * r * (n + k) > 24_000_000:
        layers = max(1, layers // 2)
    c = dict(op=op, n=n, k=k, r=r, layers=layers, grad=rng.choice(["f32", "bf16"]))
    if op == "adamw":
        c["bits"] = rng.choice([8, 32])
    return c


# --------------------------------------------------------------------------- inputs
def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _requests(case, rng):
    """(adapter or -1, tokens) of each request, in batch order: ragged lengths of at least one token that sum to m.
    Request i takes the (i mod s)-th adapter of a shuffled list; every none-th request has no adapter."""
    m, q = case["m"], min(case["requests"], case["m"])
    if q > m // 2:
        lens = [1] * q
        for i in range(m - q):
            lens[i % q] += 1
    else:
        w = [rng.random() ** 2 + 0.05 for _ in range(q)]
        lens = [1 + int((m - q) * x / sum(w)) for x in w]
        lens[rng.randrange(q)] += m - sum(lens)
    perm = list(range(case["s"]))
    rng.shuffle(perm)
    none = case["none"]
    return [(-1 if none and i % none == none - 1 else perm[i % case["s"]], n) for i, n in enumerate(lens)]


def _index(case, seed):
    req = _requests(case, random.Random(seed))
    return torch.repeat_interleave(torch.tensor([a for a, _ in req], dtype=torch.int32), torch.tensor([n for _, n in req]))


def _groups(idx, s):
    """order, offsets of the tokens sorted by adapter, tokens without one last."""
    key = torch.where(idx < 0, s, idx).long()
    order = torch.sort(key, stable=True).indices.to(torch.int32)
    counts = torch.bincount(key, minlength=s + 1)[:s]
    offsets = torch.zeros(s + 1, dtype=torch.int32)
    offsets[1:] = torch.cumsum(counts, 0)
    return order, offsets


def _shapes(case):
    """(A, B) shapes of the adapters of `layers` linear layers [n, k]."""
    return [(case["r"], case["k"]), (case["n"], case["r"])] * case["layers"]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(shape, std, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    st = {"case": case}
    if case["op"] == "groups":
        st["idx"] = _index(case, seed).cuda()
        if own:  # the scratch that a serving loop keeps
            from bit_nf4_quantized_27_b200 import binding as bd
            st["ws"] = bd.new_workspace(bd.STATUS_BYTES)
        return st
    if case["op"] in ("fwd", "bwd"):
        m, n, k, r, s = (case[x] for x in ("m", "n", "k", "r", "s"))
        idx = _index(case, seed)
        order, offsets = _groups(idx, s)
        # the adapters that have tokens, with their ranges of `order`
        st["present"] = [(a, lo, hi) for a, (lo, hi) in enumerate(zip(offsets.tolist()[:-1], offsets.tolist()[1:])) if hi > lo]
        st["idx"], st["order"], st["offsets"] = idx.cuda(), order.cuda(), offsets.cuda()
        st["X"] = normal((m, k), 1.0)
        st["A"] = normal((s, r, k), k ** -0.5)
        st["B"] = normal((s, n, r), 0.05)
        st["scales"] = 1.0 + torch.rand(s, generator=g, device="cuda")  # alpha / r between 1 and 2
        ranks = [r] * s
        if case["mixed"]:  # adapters of lower rank in slots of rank r
            rng = random.Random(seed + 1)
            ranks = [8 * rng.randint(1, r // 8) for _ in range(s)]
        st["rank_list"] = ranks
        st["ranks"] = torch.tensor(ranks, dtype=torch.int32, device="cuda")
        if case["op"] == "fwd":
            st["Y"] = normal((m, n), 1.0, _dtype(case["out"]))  # the shared projection's output
        else:
            st["dY"] = normal((m, n), 1.0)
            st["dX"] = normal((m, k), 1.0, _dtype(case["out"]))  # the shared projection's input gradient
            st["dA"] = torch.empty(s, r, k, dtype=_dtype(case["out"]), device="cuda")
            st["dB"] = torch.empty(s, n, r, dtype=_dtype(case["out"]), device="cuda")
        if own:
            from bit_nf4_quantized_27_b200 import binding as bd
            st["pool"] = bd.AdapterPool(st["A"], st["B"], st["scales"], st["ranks"] if case["mixed"] else None)
            st["ws"] = bd.new_workspace(bd.workspace_bytes_adapters(m, n, k, r, case["op"] == "bwd"))
        return st
    # a list of tensors, each starting at a multiple of BLOCK elements of one buffer
    shapes = _shapes(case)
    sizes = [a * b for a, b in shapes]
    starts, at = [], 0
    for z in sizes:
        starts.append(at)
        at += -(-z // BLOCK) * BLOCK
    nb = at // BLOCK
    blocks = torch.tensor([-(-z // BLOCK) for z in sizes])
    live = torch.ones(at, dtype=torch.bool, device="cuda")
    for z, o in zip(sizes, starts):
        if z % BLOCK:
            live[o + z:o + -(-z // BLOCK) * BLOCK] = False
    st["grad"] = (normal((at,), 1e-3, torch.float32) * live).to(_dtype(case["grad"]))

    def views(flat):
        return [flat[o:o + z] for z, o in zip(sizes, starts)]

    if case["op"] == "norm":
        if own:
            from bit_nf4_quantized_27_b200 import binding as bd
            st["list"] = bd.TensorList(grads=views(st["grad"]))
            st["ws"] = bd.new_workspace(bd.workspace_bytes_grad_norm())
        return st
    st["p"] = normal((at,), 0.05, torch.float32) * live
    st["p16"] = st["p"].to(torch.bfloat16)
    st["clip"] = torch.tensor([1.0, 0.75], device="cuda")
    # B matrices learn sixteen times as fast as A
    st["lr_scales"] = [1.0, 16.0] * case["layers"]
    st["lr_scale"] = torch.repeat_interleave(torch.tensor(st["lr_scales"]), blocks).cuda().view(nb, 1)
    first = torch.repeat_interleave(torch.cumsum(blocks, 0) - blocks, blocks)
    st["block_in_tensor"] = (torch.arange(nb) - first).cuda().view(nb, 1)
    st["tensor_of_block"] = torch.repeat_interleave(torch.arange(len(sizes)), blocks).cuda().view(nb, 1)
    # states as after some steps: momentum about the gradients' size, variance about their squares
    m = normal((at,), 3e-4, torch.float32) * live
    v = (normal((at,), 1e-3, torch.float32) ** 2 + 1e-8) * live
    if case["bits"] == 32:
        st["m"], st["v"] = m, v
    else:
        m, v = m.view(nb, BLOCK), v.view(nb, BLOCK)
        st["ms"], st["vs"] = m.abs().amax(1) / 448.0, v.amax(1) / 57344.0
        st["m"] = (m / st["ms"].clamp(min=1e-30)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(-1)
        st["v"] = (v / st["vs"].clamp(min=1e-30)[:, None]).clamp(0, 57344).to(torch.float8_e5m2).view(-1)
    if own:
        from bit_nf4_quantized_27_b200 import binding as bd
        scale_views = {}
        if case["bits"] == 8:
            sv = lambda flat: [flat[o // BLOCK:o // BLOCK + -(-z // BLOCK)] for z, o in zip(sizes, starts)]  # noqa: E731
            scale_views = dict(exp_avg_scale=sv(st["ms"]), exp_avg_sq_scale=sv(st["vs"]))
        st["list"] = bd.TensorList(params=views(st["p"]), p_bf16=views(st["p16"]), grads=views(st["grad"]),
                                   exp_avg=views(st["m"]), exp_avg_sq=views(st["v"]), lr_scale=st["lr_scales"], **scale_views)
    return st


# --------------------------------------------------------------------------- one pass
def run(st):
    return {"groups": _run_groups, "fwd": _run_fwd, "bwd": _run_bwd, "norm": _run_norm, "adamw": _run_adamw}[st["case"]["op"]](st)


def _run_groups(st):
    s = st["case"]["s"]
    if own:
        from bit_nf4_quantized_27_b200 import binding as bd
        return bd.adapter_groups(st["idx"], s, ws=st["ws"])
    key = torch.where(st["idx"] < 0, s, st["idx"])
    order = torch.sort(key, stable=True).indices.to(torch.int32)
    counts = torch.bincount(key, minlength=s + 1)
    offsets = torch.cumsum(counts, 0)[:s].to(torch.int32)
    return order, torch.cat([offsets.new_zeros(1), offsets])


def _run_fwd(st):
    if own:
        from bit_nf4_quantized_27_b200 import binding as bd
        bd.adapters_fwd(st["pool"], (st["order"], st["offsets"]), st["X"], st["Y"], ws=st["ws"])
        return st["Y"]
    X, Y, A, B = st["X"], st["Y"], st["A"], st["B"]
    if len(X) <= 64:  # few tokens: one batched product, each token with its own adapter
        at = st["idx"].clamp(min=0).long()
        scale = torch.where(st["idx"] < 0, 0.0, st["scales"][at])[:, None]
        t = torch.bmm(A[at].float(), X.float()[:, :, None])[:, :, 0]
        t = torch.where(torch.arange(t.shape[1], device="cuda") < st["ranks"][at][:, None], t, 0.0)
        Y.copy_(Y.float() + scale * torch.bmm(B[at].float(), t[:, :, None])[:, :, 0])
        return Y
    for a, lo, hi in st["present"]:  # one product a request's adapter: a padded batch of all of them would be larger
        rows, rk = st["order"][lo:hi], st["rank_list"][a]
        t = X[rows].float() @ A[a, :rk].float().t()
        Y[rows] = (Y[rows].float() + st["scales"][a] * (t @ B[a, :, :rk].float().t())).to(Y.dtype)
    return Y


def _run_bwd(st):
    if own:
        from bit_nf4_quantized_27_b200 import binding as bd
        bd.adapters_bwd(st["pool"], (st["order"], st["offsets"]), st["X"], st["dY"], dX=st["dX"], outs=(st["dA"], st["dB"]),
                        ws=st["ws"])
        return {"dX": st["dX"], "dA": st["dA"], "dB": st["dB"]}
    X, dY, dX, A, B = st["X"], st["dY"], st["dX"], st["A"], st["B"]
    dA, dB = st["dA"].zero_(), st["dB"].zero_()
    for a, lo, hi in st["present"]:
        rows, rk, s = st["order"][lo:hi], st["rank_list"][a], st["scales"][a]
        Af, Bf, x, dy = A[a, :rk].float(), B[a, :, :rk].float(), X[rows].float(), dY[rows].float()
        t, u = x @ Af.t(), s * (dy @ Bf)
        dX[rows] = (dX[rows].float() + u @ Af).to(dX.dtype)
        dA[a, :rk] = (u.t() @ x).to(dA.dtype)
        dB[a, :, :rk] = (s * (dy.t() @ t)).to(dB.dtype)
    return {"dX": dX, "dA": dA, "dB": dB}


def _run_norm(st):
    if own:
        from bit_nf4_quantized_27_b200 import binding as bd
        return bd.grad_norm(st["list"], 0.3, ws=st["ws"])
    norm = st["grad"].double().square().sum().sqrt()
    return torch.stack([norm, (0.3 / (norm + 1e-6)).clamp(max=1.0)]).float()


def _f32(x):
    """A hyper-parameter as the float32 that the step is given."""
    return float(torch.tensor(x, dtype=torch.float32))


def _hash(st, nb):
    """32 random-looking bits for each element, from (seed, tensor, place in the tensor)."""
    mask = 0xFFFFFFFF
    e = st["block_in_tensor"] * BLOCK + torch.arange(BLOCK, device="cuda")
    x = ((e + STEP * 0xB7E15163 + st["tensor_of_block"] * 0x3504F333) * 0x9E3779B9) & mask
    x = ((x ^ (x >> 16)) * 0x6A09E667) & mask
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & mask
    return x ^ (x >> 16)


def _round8(x, rnd, drop, least, most):
    """x >= 0 rounded down or up to a float8 value: `drop` float32 mantissa bits go, after `rnd` (that many bits) is added to them; below the
    least normal value the step is the same as just above it."""
    small = x < least
    z = torch.where(small, x + least, x)
    z = ((z.view(torch.int32) + rnd.to(torch.int32)) & -(1 << drop)).view(torch.float32)
    return torch.where(small, z - least, z).clamp(max=most)


def _run_adamw(st):
    c = st["case"]
    if own:
        from bit_nf4_quantized_27_b200 import binding as bd
        bd.adamw_multi(st["list"], STEP, clip=st["clip"], seed=STEP, **HYPER)
    else:
        h = {k: _f32(v) for k, v in HYPER.items()}
        nb = st["p"].numel() // BLOCK
        p, g = st["p"].view(nb, BLOCK), st["grad"].view(nb, BLOCK).float() * st["clip"][1]
        if c["bits"] == 32:
            m, v = st["m"].view(nb, BLOCK), st["v"].view(nb, BLOCK)
        else:
            m = st["m"].view(nb, BLOCK).float() * st["ms"][:, None]
            v = st["v"].view(nb, BLOCK).float() * st["vs"][:, None]
        lr = h["lr"] * st["lr_scale"].double()
        bc1, bc2 = 1.0 - h["beta1"] ** STEP, 1.0 - h["beta2"] ** STEP
        decay, step_size = (1.0 - lr * h["weight_decay"]).float(), (lr / bc1).float()
        m = m * h["beta1"] + g * (1.0 - h["beta1"])
        v = v * h["beta2"] + (g * g) * (1.0 - h["beta2"])
        denom = v.sqrt() / math.sqrt(bc2) + h["eps"]
        p.copy_(p * decay - (step_size * m) / denom)
        st["p16"].view(nb, BLOCK).copy_(p)
        if c["bits"] == 32:
            st["m"].view(nb, BLOCK).copy_(m)
            st["v"].view(nb, BLOCK).copy_(v)
        else:
            bits = _hash(st, nb)
            mm, vm = m.abs().amax(1, keepdim=True), v.amax(1, keepdim=True)
            qm = _round8(m.abs() * torch.where(mm > 0, 448.0 / mm, 0.0), bits & 0xFFFFF, 20, 2.0 ** -6, 448.0)
            qv = _round8(v * torch.where(vm > 0, 57344.0 / vm, 0.0), bits >> 11, 21, 2.0 ** -14, 57344.0)
            qv = torch.where(v > 0, qv.clamp(min=2.0 ** -16), qv)  # a variance that is not zero stays above zero
            st["m"].view(nb, BLOCK).copy_(torch.copysign(qm, m).to(torch.float8_e4m3fn))
            st["v"].view(nb, BLOCK).copy_(qv.to(torch.float8_e5m2))
            st["ms"].copy_((mm / 448.0).view(-1))
            st["vs"].copy_((vm / 57344.0).view(-1))
    out = {"p": st["p"], "p16": st["p16"], "m": st["m"], "v": st["v"]}
    return out if c["bits"] == 32 else {**out, "m_scale": st["ms"], "v_scale": st["vs"]}


# --------------------------------------------------------------------------- what a pass needs
def work(case):
    op = case["op"]
    if op == "groups":
        return {"bytes": 8 * case["m"] + 4 * (case["s"] + 1), "flops": 0}
    if op in ("fwd", "bwd"):
        m, n, k, r = (case[x] for x in ("m", "n", "k", "r"))
        req = _requests(case, random.Random(0))
        rows, used = sum(c for a, c in req if a >= 0), len({a for a, _ in req if a >= 0})
        r_mean = (8 + r) / 2 if case["mixed"] else r
        e = 4 if case["out"] == "f32" else 2
        pool = used * r_mean * (n + k) * 2
        if op == "fwd":
            return {"bytes": rows * (2 * k + 2 * e * n) + pool, "flops": 2 * rows * r_mean * (n + k)}
        return {"bytes": rows * (2 * k + 2 * n + 2 * e * k) + pool + e * case["s"] * r * (n + k),
                "flops": rows * r_mean * (4 * (n + k) + 2 * k)}
    n = case["layers"] * case["r"] * (case["n"] + case["k"])
    g = 4 if case["grad"] == "f32" else 2
    if op == "norm":
        return {"bytes": n * g, "flops": 2 * n}
    return {"bytes": n * (8 + 2 + g + (16 if case["bits"] == 32 else 4 + 16 / BLOCK)), "flops": 14 * n}


# --------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "groups":
        return None
    if op in ("fwd", "bwd"):
        idx, X = st["idx"].long(), st["X"].double()
        m, r, s = case["m"], case["r"], case["s"]
        keep = torch.arange(r, device="cuda") < st["ranks"][:, None]  # [s, r]
        A = torch.where(keep[:, :, None], st["A"].double(), 0.0)
        B = torch.where(keep[:, None, :], st["B"].double(), 0.0)
        sc = st["scales"].double()
        if op == "fwd":
            Y = st["Y"].double()
            for a in range(s):
                at = torch.nonzero(idx == a).view(-1)
                Y.index_add_(0, at, sc[a] * torch.einsum("mr,nr->mn", torch.einsum("mk,rk->mr", X[at], A[a]), B[a]))
            return Y
        dY, dX, dA, dB = st["dY"].double(), st["dX"].double(), torch.zeros_like(A), torch.zeros_like(B)
        for a in range(s):
            at = torch.nonzero(idx == a).view(-1)
            U = torch.einsum("mn,nr->mr", dY[at], B[a]) * sc[a]
            dX.index_add_(0, at, torch.einsum("mr,rk->mk", U, A[a]))
            dA[a] = torch.einsum("mr,mk->rk", U, X[at])
            dB[a] = sc[a] * torch.einsum("mn,mr->nr", dY[at], torch.einsum("mk,rk->mr", X[at], A[a]))
        return {"dX": dX, "dA": dA, "dB": dB}
    if op == "norm":
        n = torch.linalg.vector_norm(st["grad"].double())
        return torch.stack([n, torch.minimum(torch.ones_like(n), 0.3 / (n + 1e-6))])
    # AdamW: the step in the order of its formula, then the states' scales and codes
    h = {k: _f32(v) for k, v in HYPER.items()}
    nb = st["p"].numel() // BLOCK
    p, m, v = (st[x].double().view(nb, BLOCK) for x in ("p", "m", "v"))
    if case["bits"] == 8:
        m, v = m * st["ms"].double()[:, None], v * st["vs"].double()[:, None]
    g = st["grad"].double().view(nb, BLOCK) * st["clip"][1].double()
    lr = h["lr"] * st["lr_scale"].double()
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g ** 2
    mhat, vhat = m / (1 - h["beta1"] ** STEP), v / (1 - h["beta2"] ** STEP)
    p = p - lr * h["weight_decay"] * p - lr * mhat / (torch.sqrt(vhat) + h["eps"])
    out = {"p": p.view(-1), "p16": p.view(-1)}
    if case["bits"] == 32:
        return {**out, "m": m.view(-1), "v": v.view(-1)}

    def code(x, u, mantissa, lowest, most):
        x = x / x.amax(1, keepdim=True).clamp(min=1e-300) * most
        step = torch.exp2(((torch.frexp(x).exponent - 1).clamp(min=lowest) - mantissa).double())
        return (torch.floor(x / step + u) * step).clamp(max=most)

    rnd = _hash(st, nb)
    qm, qv = code(m.abs(), (rnd & 0xFFFFF) / 2.0 ** 20, 3, -6, 448.0), code(v, (rnd >> 11) / 2.0 ** 21, 2, -14, 57344.0)
    qv = torch.where(v > 0, qv.clamp(min=2.0 ** -16), qv)
    return {**out, "m": (qm * m.sign()).view(-1), "v": qv.view(-1), "m_scale": m.abs().amax(1) / 448, "v_scale": v.amax(1) / 57344}
