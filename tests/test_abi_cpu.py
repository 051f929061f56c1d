"""The C-ABI library loads, exports every declared symbol, and its host-side
logic (sizes, table, argument checks) behaves without a GPU."""

import ctypes

import numpy as np
import pytest

import oracle as O
from bit_nf4_quantized_27_b200 import binding as bd
from bit_nf4_quantized_27_b200.build import build


@pytest.fixture(scope="module")
def L():
    build()
    return bd.lib()


def test_exports_every_declared_symbol(L):
    names = bd.header_functions()
    assert len(names) >= 10
    for n in names:
        assert hasattr(L, n), n


def test_abi_version(L):
    assert L.qlora_abi_version() == 2


def test_codebook_equals_oracle_bit_for_bit(L):
    got = np.array(bd.codebook(), dtype=np.float32)
    assert np.array_equal(got.view(np.uint32), O.nf4_levels().view(np.uint32))


@pytest.mark.parametrize("rows,cols", [(256, 256), (4096, 4096), (11008, 4096), (3, 64), (1, 64 * 300)])
def test_storage_bytes_match_oracle(L, rows, cols):
    total, c, s, g = bd.storage_bytes(rows, cols)
    oc, os_, og = O.storage_bytes(rows, cols)
    assert (c, s, g) == (oc, os_, og) and total == c + s + g


def test_storage_bytes_rejects_bad_cols(L):
    assert bd.storage_bytes(4, 65)[0] == 0
    assert bd.storage_bytes(0, 64)[0] == 0


def test_workspace_bytes(L):
    assert bd.workspace_bytes(16, 11008, 4096, 64, False) >= 256 + 16 * 64 * 2
    assert bd.workspace_bytes(2048, 4096, 4096, 64, True) >= 256 + 2 * 2048 * 64 * 2
    assert bd.workspace_bytes(0, 1, 64, 8, False) == 0
    assert bd.workspace_bytes(1, 1, 64, 512, False) == 0


def _t(rows, cols, codes=0x1000, sc=0x2000, c2=0x3000):
    return bd.NF4TensorC(rows, cols, codes, sc, c2)


def test_argument_checks_without_gpu(L):
    # Every check runs before any device work; fake (never dereferenced) pointers.
    W, ws = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000)
    good = _t(64, 64)
    assert L.qlora_nf4_quantize(W, 1, ctypes.byref(_t(64, 65)), ws, None) == 2
    assert L.qlora_nf4_quantize(W, 1, ctypes.byref(_t(64, 64, codes=0)), ws, None) == 1
    assert L.qlora_nf4_quantize(None, 1, ctypes.byref(good), ws, None) == 1
    assert L.qlora_nf4_quantize(W, 7, ctypes.byref(good), ws, None) == 1
    assert L.qlora_nf4_quantize(ctypes.c_void_p(0x10008), 1, ctypes.byref(good), ws, None) == 3
    assert L.qlora_nf4_quantize(W, 1, ctypes.byref(_t(64, 64, codes=0x1004)), ws, None) == 3
    bad_fmt = _t(64, 64)
    bad_fmt.scale_format = 3
    assert L.qlora_nf4_quantize(W, 1, ctypes.byref(bad_fmt), ws, None) == 1
    bad_fmt.scale_format = -1
    assert L.qlora_nf4_dequantize(ctypes.byref(bad_fmt), ws, 1, None) == 1
    ad = bd.LoraC(64, 16.0, 0x4000, 0x5000)
    X, Y = ctypes.c_void_p(0x6000), ctypes.c_void_p(0x7000)
    assert L.qlora_linear_fwd(ctypes.byref(good), ctypes.byref(bd.LoraC(12, 16.0, 0x4000, 0x5000)), X, 4, Y, 1,
                              None, ws, 1 << 20, None) == 1
    assert L.qlora_linear_fwd(ctypes.byref(good), ctypes.byref(ad), X, 0, Y, 1, None, ws, 1 << 20, None) == 1
    assert L.qlora_linear_fwd(ctypes.byref(good), ctypes.byref(ad), X, 4, Y, 1, None, ws, 16, None) == 4
    assert L.qlora_linear_fwd(ctypes.byref(_t(60, 64)), ctypes.byref(ad), X, 4, Y, 1, None, ws, 1 << 20, None) == 2
    assert L.qlora_linear_bwd(ctypes.byref(good), ctypes.byref(ad), X, None, 4, None, X, 1, X, X, 1, ws, 1 << 20,
                              None) == 1


def test_valid_call_without_gpu_reports_no_device(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    W, ws = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000)
    assert L.qlora_nf4_quantize(W, 1, ctypes.byref(_t(64, 64)), ws, None) == 8


def test_selftest_argument_checks_without_gpu(L):
    ws = ctypes.c_void_p(0x20000)
    assert L.qlora_selftest_bounded_wait(None, 1000, None) == 1
    assert L.qlora_selftest_bounded_wait(ws, 0, None) == 1
    assert L.qlora_selftest_bounded_wait(ws, 2000001, None) == 1
    assert L.qlora_selftest_bounded_wait(ctypes.c_void_p(0x20010), 1000, None) == 3
    import torch
    if not torch.cuda.is_available():
        assert L.qlora_selftest_bounded_wait(ws, 1000, None) == 8


def test_status_strings(L):
    for code in range(9):
        assert L.qlora_status_string(code)
    assert L.qlora_status_string(0) == b"ok"


def test_device_level_literals_match_bit_patterns():
    # the kernels use the 16 levels both as float32 bit patterns and as hex-float
    # immediates; both lists, and the oracle's table, must be identical
    import os
    import re
    import struct

    src = open(os.path.join(os.path.dirname(bd.LIB_PATH), "csrc", "nf4_device.cuh")).read()
    bits_block = src[src.index("kNf4LevelBits[16] = {"):]
    bits = [int(b, 16) for b in re.findall(r"0x([0-9a-f]{8})u", bits_block[:bits_block.index("};")])]
    fn = src[src.index("constexpr float nf4_level(int j)"):]
    fn = fn[:fn.index("}")]
    lits = re.findall(r"(-?0x[0-9a-f.]+p[+-]\d+)f", fn)
    vals = [struct.unpack("<I", struct.pack("<f", float.fromhex(v)))[0] for v in lits]
    assert len(bits) == 16 and len(vals) == 16
    assert bits == vals
    assert bits == [int(x) for x in O.nf4_levels().view(np.uint32)]


def test_merge_and_adamw_argument_checks_without_gpu(L):
    good = _t(64, 64)
    ad = bd.LoraC(64, 16.0, 0x4000, 0x5000)
    out = ctypes.c_void_p(0x6000)
    assert L.qlora_lora_merge(ctypes.byref(good), ctypes.byref(ad), None, None) == 1
    assert L.qlora_lora_merge(ctypes.byref(good), ctypes.byref(ad), ctypes.c_void_p(0x6008), None) == 3
    assert L.qlora_lora_merge(ctypes.byref(good), ctypes.byref(bd.LoraC(12, 16.0, 0x4000, 0x5000)), out, None) == 1
    assert L.qlora_lora_merge(ctypes.byref(_t(64, 65)), ctypes.byref(ad), out, None) == 2
    p, g, m, v, h = (ctypes.c_void_p(a) for a in (0x10000, 0x20000, 0x30000, 0x40000, 0x50000))
    hp = bd.AdamWC(1e-3, 0.9, 0.999, 1e-8, 0.01)
    assert L.qlora_adamw_step(p, h, g, m, v, 0, ctypes.byref(hp), 1, None) == 1
    assert L.qlora_adamw_step(p, h, g, m, v, 10, ctypes.byref(hp), 0, None) == 1
    assert L.qlora_adamw_step(p, h, g, m, v, 10, ctypes.byref(bd.AdamWC(1e-3, 1.0, 0.999, 1e-8, 0.0)), 1, None) == 1
    assert L.qlora_adamw_step(p, h, g, m, v, 10, ctypes.byref(bd.AdamWC(1e-3, 0.9, 0.999, 0.0, 0.0)), 1, None) == 1
    assert L.qlora_adamw_step(p, h, None, m, v, 10, ctypes.byref(hp), 1, None) == 1
    assert L.qlora_adamw_step(ctypes.c_void_p(0x10004), h, g, m, v, 10, ctypes.byref(hp), 1, None) == 3
    assert L.qlora_adamw_step(p, ctypes.c_void_p(0x50002), g, m, v, 10, ctypes.byref(hp), 1, None) == 3
    import torch
    if not torch.cuda.is_available():
        assert L.qlora_adamw_step(p, None, g, m, v, 10, ctypes.byref(hp), 1, None) == 8
        assert L.qlora_lora_merge(ctypes.byref(good), ctypes.byref(ad), out, None) == 8


def test_multi_adapter_argument_checks_without_gpu(L):
    good = _t(1024, 1024)
    ads = (bd.LoraC * 2)(bd.LoraC(16, 16.0, 0x4000, 0x5000), bd.LoraC(16, 8.0, 0x6000, 0x7000))
    idx = (ctypes.c_int32 * 3)(0, 1, 1)
    X, Y, ws = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000), ctypes.c_void_p(0x30000)
    f = L.qlora_linear_fwd_multi
    assert f(ctypes.byref(good), ads, 2, idx, X, 3, Y, 1, ws, 1 << 20, None) in (0, 8)  # valid (no GPU: 8)
    bad_idx = (ctypes.c_int32 * 3)(0, 2, 1)
    assert f(ctypes.byref(good), ads, 2, bad_idx, X, 3, Y, 1, ws, 1 << 20, None) == 1
    assert f(ctypes.byref(good), ads, 2, idx, X, 17, Y, 1, ws, 1 << 20, None) == 1
    assert f(ctypes.byref(good), ads, 0, idx, X, 3, Y, 1, ws, 1 << 20, None) == 1
    mixed = (bd.LoraC * 2)(bd.LoraC(16, 16.0, 0x4000, 0x5000), bd.LoraC(32, 8.0, 0x6000, 0x7000))
    assert f(ctypes.byref(good), mixed, 2, idx, X, 3, Y, 1, ws, 1 << 20, None) == 1
    assert f(ctypes.byref(_t(1024, 576)), ads, 2, idx, X, 3, Y, 1, ws, 1 << 20, None) == 2
    assert f(ctypes.byref(good), ads, 2, idx, X, 3, Y, 1, ws, 64, None) == 4


def test_dropout_argument_checks_without_gpu(L):
    good = _t(64, 64)
    ad = bd.LoraC(64, 16.0, 0x4000, 0x5000)
    X, keep, Y, ws = (ctypes.c_void_p(a) for a in (0x10000, 0x20000, 0x30000, 0x40000))
    f = L.qlora_linear_fwd_dropout
    big = 1 << 24
    assert f(ctypes.byref(good), ctypes.byref(ad), X, keep, 1.0, 32, Y, 1, None, ws, big, None) == 1
    assert f(ctypes.byref(good), ctypes.byref(ad), X, keep, -0.1, 32, Y, 1, None, ws, big, None) == 1
    assert f(ctypes.byref(good), ctypes.byref(ad), X, None, 0.1, 32, Y, 1, None, ws, big, None) == 1
    assert f(ctypes.byref(good), ctypes.byref(ad), X, ctypes.c_void_p(0x20008), 0.1, 32, Y, 1, None, ws, big,
             None) == 3
    assert f(ctypes.byref(good), ctypes.byref(ad), X, keep, 0.1, 32, Y, 1, None, ws, 64, None) == 4
    b = L.qlora_linear_bwd_dropout
    dX, dA, dB = (ctypes.c_void_p(a) for a in (0x50000, 0x60000, 0x70000))
    assert b(ctypes.byref(good), ctypes.byref(ad), X, X, keep, 1.5, 32, None, dX, 1, dA, dB, 1, ws, big, None) == 1
    assert b(ctypes.byref(good), ctypes.byref(ad), X, X, None, 0.1, 32, None, dX, 1, dA, dB, 1, ws, big, None) == 1
    # the dropout workspace holds the masked copy of X on top of the plain one
    for bwd in (0, 1):
        assert L.qlora_workspace_bytes_dropout(300, 512, 1024, 64, bwd) >= \
            L.qlora_workspace_bytes(300, 512, 1024, 64, bwd) + 300 * 1024 * 2


def test_keep_mask_generator_packs_like_the_oracle():
    import numpy as np
    import torch

    from bit_nf4_quantized_27_b200 import inputs as I

    packed = I.keep_mask(5, 48, 0.3, 11)
    assert packed.dtype == torch.uint8 and tuple(packed.shape) == (5, 6)
    g = torch.Generator().manual_seed(11)
    want = (torch.rand((5, 48), generator=g, dtype=torch.float64) >= 0.3).numpy()
    assert np.array_equal(O.unpack_keep(packed.numpy(), 5, 48), want)


def test_multi_workspace_size(L):
    for m, n, k, r in ((1, 11008, 4096, 64), (16, 11008, 4096, 64), (7, 1000, 512, 24)):
        lo = L.qlora_workspace_bytes(m, n, k, r, 0)
        assert L.qlora_workspace_bytes_multi(m, n, k, r) == lo + ((m * n * 4 + 255) // 256) * 256
    assert L.qlora_workspace_bytes_multi(17, 1024, 1024, 16) == 0
    assert L.qlora_workspace_bytes_multi(4, 1024, 1024, 300) == 0


def _pool(n=4, r=16, A=0x4000, B=0x5000, ranks=None, scales=0x6000):
    return bd.PoolC(n, r, A, B, ranks, scales)


def test_adapter_groups_argument_checks_without_gpu(L):
    idx, order, off, ws = (ctypes.c_void_p(a) for a in (0x10000, 0x20000, 0x30000, 0x40000))
    f = L.qlora_adapter_groups
    assert f(idx, -1, 4, order, off, ws, None) == 1
    assert f(idx, 10, 0, order, off, ws, None) == 1
    assert f(idx, 10, 1025, order, off, ws, None) == 1
    assert f(None, 10, 4, order, off, ws, None) == 1
    assert f(idx, 10, 4, order, None, ws, None) == 1
    assert f(idx, 10, 4, order, off, None, None) == 1
    assert f(ctypes.c_void_p(0x10002), 10, 4, order, off, ws, None) == 3
    assert f(idx, 10, 4, order, off, ctypes.c_void_p(0x40010), None) == 3


def test_adapters_argument_checks_without_gpu(L):
    order, off, X, Y, T, ws = (0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000)
    big = 1 << 24

    def fwd(pool=None, order=order, off=off, X=X, ldx=128, M=10, N=64, K=128, Y=Y, ldy=64, dt=1, T=T, ws=ws, size=big):
        pool = _pool() if pool is None else pool
        return L.qlora_adapters_fwd(ctypes.byref(pool), order, off, X, ldx, M, N, K, Y, ldy, dt, T, ws, size, None)

    import torch
    if not torch.cuda.is_available():
        assert fwd() == 8 and fwd(T=None) == 8 and fwd(M=0, X=None, order=None, Y=None) == 8
    for bad in (_pool(n=0), _pool(n=1025), _pool(r=12), _pool(r=0), _pool(r=264), _pool(A=None), _pool(B=None), _pool(scales=None)):
        assert fwd(pool=bad) == 1
    for bad in (_pool(A=0x4008), _pool(B=0x5008), _pool(ranks=0x7002)):
        assert fwd(pool=bad) == 3
    assert fwd(order=None) == 1 and fwd(off=None) == 1 and fwd(X=None) == 1 and fwd(Y=None) == 1 and fwd(ws=None) == 1
    assert fwd(M=-1) == 1 and fwd(M=1 << 29) == 1 and fwd(dt=2) == 1
    assert fwd(K=124, ldx=128) == 2 and fwd(N=60) == 2 and fwd(N=0) == 2 and fwd(ldx=120) == 2 and fwd(ldx=132) == 2
    assert fwd(ldy=63) == 2
    assert fwd(X=X + 8) == 3 and fwd(Y=Y + 1) == 3 and fwd(Y=Y + 2, dt=0) == 3 and fwd(T=T + 8) == 3 and fwd(ws=ws + 16) == 3
    assert fwd(size=L.qlora_workspace_bytes_adapters(10, 64, 128, 16, 0) - 1) == 4
    dY, dX, dA, dB = 0x70000, 0x80000, 0x90000, 0xa0000

    def bwd(pool=None, X=X, ldx=128, dY=dY, lddy=64, M=10, N=64, K=128, T=T, dX=dX, lddx=128, xdt=1, dA=dA, dB=dB, gdt=0,
            ws=ws, size=big):
        pool = _pool() if pool is None else pool
        return L.qlora_adapters_bwd(ctypes.byref(pool), order, off, X, ldx, dY, lddy, M, N, K, T, dX, lddx, xdt, dA, dB, gdt, ws,
                                    size, None)

    if not torch.cuda.is_available():
        assert bwd() == 8 and bwd(dX=None, lddx=0) == 8 and bwd(dA=None, dB=None) == 8 and bwd(T=None) == 8
    assert bwd(dY=None) == 1 and bwd(dA=None) == 1 and bwd(dB=None) == 1 and bwd(gdt=3) == 1 and bwd(xdt=3) == 1
    assert bwd(lddy=60) == 2 and bwd(lddy=68) == 2 and bwd(lddx=120) == 2
    assert bwd(dY=dY + 8) == 3 and bwd(dX=dX + 1) == 3 and bwd(dA=dA + 4) == 3 and bwd(dB=dB + 4) == 3
    assert bwd(size=L.qlora_workspace_bytes_adapters(10, 64, 128, 16, 1) - 1) == 4


def test_pool_layer_argument_checks_without_gpu(L):
    order, off, X, Y, ws, big = 0x10000, 0x20000, 0x30000, 0x40000, 0x60000, 1 << 24
    f, b, p = L.qlora_linear_fwd_pool, L.qlora_linear_bwd_pool, _pool()
    good = _t(64, 128)
    assert f(ctypes.byref(_t(64, 100)), ctypes.byref(p), order, off, X, 4, Y, 1, None, ws, big, None) == 2
    assert f(ctypes.byref(_t(60, 128)), ctypes.byref(p), order, off, X, 4, Y, 1, None, ws, big, None) == 2
    assert f(ctypes.byref(good), ctypes.byref(p), order, off, X, 0, Y, 1, None, ws, big, None) == 1
    assert f(ctypes.byref(good), ctypes.byref(p), order, off, X, 4, None, 1, None, ws, big, None) == 1
    assert f(ctypes.byref(good), ctypes.byref(p), order, off, X, 4, Y, 5, None, ws, big, None) == 1
    assert f(ctypes.byref(good), ctypes.byref(p), order, off, X, 4, Y + 8, 1, None, ws, big, None) == 3
    assert f(ctypes.byref(good), ctypes.byref(p), order, off, X, 4, Y, 1, None, ws, 64, None) == 4
    assert b(ctypes.byref(good), ctypes.byref(p), order, off, X, Y, 4, None, None, 1, Y, Y, 1, ws, big, None) == 1
    assert b(ctypes.byref(good), ctypes.byref(p), order, off, X, Y, 4, None, Y, 1, Y, Y, 7, ws, big, None) == 1
    assert b(ctypes.byref(good), ctypes.byref(p), order, off, X, Y, 4, None, Y, 1, Y + 8, Y, 1, ws, big, None) == 3
    assert b(ctypes.byref(good), ctypes.byref(p), order, off, X, Y, 4, None, Y, 1, Y, Y, 1, ws, 64, None) == 4


def test_adapters_workspace_size(L):
    f = L.qlora_workspace_bytes_adapters
    assert f(10, 64, 128, 16, 0) == 256 + 1024 and f(10, 64, 128, 16, 1) == 256 + 2 * 1024
    assert f(0, 64, 128, 16, 1) == 256
    assert f(-1, 64, 128, 16, 0) == 0 and f(1, 64, 128, 12, 0) == 0 and f(1, 64, 128, 264, 0) == 0 and f(1, 0, 128, 8, 0) == 0


def _tensor(n=100, grad=0x1000, p=0x2000, p16=0x3000, m=0x4000, v=0x5000, ms=0x6000, vs=0x7000, lr=1.0):
    return bd.TensorC(n, grad, p, p16, m, v, ms, vs, lr)


def test_tensor_list_argument_checks_without_gpu(L):
    import torch
    table, out = 0x100000, bd.TensorListC()

    def init(t, bits=32, gdt=0, n=1, table=table, size=1 << 20):
        return L.qlora_tensor_list_init((bd.TensorC * 1)(t), n, gdt, bits, table, size, ctypes.byref(out), None)

    assert init(_tensor(), n=0) == 1 and init(_tensor(), bits=16) == 1 and init(_tensor(), gdt=2) == 1
    assert init(_tensor(), table=None) == 1 and init(_tensor(n=-1)) == 2 and init(_tensor(n=1 << 50)) == 2
    assert init(_tensor(), table=table + 8) == 3 and init(_tensor(), size=8) == 4
    assert init(_tensor(grad=None)) == 1 and init(_tensor(p=None)) == 1 and init(_tensor(m=None)) == 1
    assert init(_tensor(lr=-1.0)) == 1 and init(_tensor(lr=float("nan"))) == 1
    assert init(_tensor(ms=None), bits=8) == 1 and init(_tensor(vs=None), bits=8) == 1
    assert init(_tensor(grad=0x1002)) == 3 and init(_tensor(p=0x2002)) == 3 and init(_tensor(m=0x4001)) == 3
    if not torch.cuda.is_available():
        assert init(_tensor()) == 8 and init(_tensor(ms=None, vs=None)) == 8 and init(_tensor(m=0x4001, v=0x5003), bits=8) == 8
        assert init(_tensor(p=None, m=None, v=None), bits=0) == 8 and init(_tensor(n=0, grad=None, p=None)) == 8
    f = L.qlora_tensor_list_bytes
    one = f((bd.TensorC * 1)(_tensor(n=2048)), 1)
    assert f((bd.TensorC * 1)(_tensor(n=2049)), 1) == one + 8 and f((bd.TensorC * 1)(_tensor(n=0)), 1) == one
    assert f((bd.TensorC * 1)(_tensor(n=-1)), 1) == 0 and f(None, 1) == 0


def test_grad_norm_and_adamw_multi_argument_checks_without_gpu(L):
    import torch
    need = L.qlora_workspace_bytes_grad_norm()
    ok = bd.TensorListC(0x100000, 3, 32, 0, 10)
    norm, ws = 0x200000, 0x300000

    def gn(l=ok, most=1.0, out=norm, ws=ws, size=need):
        return L.qlora_grad_norm(ctypes.byref(l), most, out, ws, size, None)

    assert gn(bd.TensorListC(None, 3, 32, 0, 10)) == 1 and gn(bd.TensorListC(0x100000, 0, 32, 0, 10)) == 1
    assert gn(bd.TensorListC(0x100000, 3, 32, 4, 10)) == 1 and gn(bd.TensorListC(0x100008, 3, 32, 0, 10)) == 3
    assert gn(most=-1.0) == 1 and gn(most=float("nan")) == 1 and gn(out=None) == 1 and gn(ws=None) == 1
    assert gn(out=norm + 2) == 3 and gn(ws=ws + 16) == 3 and gn(size=need - 1) == 4
    hp = bd.AdamWC(1e-3, 0.9, 0.999, 1e-8, 0.01)

    def step(l=ok, hp=hp, t=1, clip=norm):
        return L.qlora_adamw_multi(ctypes.byref(l), ctypes.byref(hp), t, clip, 0, None)

    assert step(bd.TensorListC(0x100000, 3, 0, 0, 10)) == 1 and step(t=0) == 1 and step(clip=norm + 2) == 3
    for bad in ((-1.0, 0.9, 0.999, 1e-8, 0.0), (1e-3, 1.0, 0.999, 1e-8, 0.0), (1e-3, 0.9, -0.1, 1e-8, 0.0),
                (1e-3, 0.9, 0.999, 0.0, 0.0), (1e-3, 0.9, 0.999, 1e-8, -1.0), (float("inf"), 0.9, 0.999, 1e-8, 0.0)):
        assert step(hp=bd.AdamWC(*bad)) == 1
    if not torch.cuda.is_available():
        assert gn() == 8 and step() == 8 and step(clip=None) == 8


def test_state_hash_spreads_bits():
    """Each bit of the 8-bit states' random numbers is set in about half of the elements (6 standard
    deviations), and neighbours in place, tensor and seed share about half of their bits."""
    from oracle import many_adapters as MA

    n = 20000
    x = MA.state_hash(range(n), 3, 17)
    bits = lambda v: np.unpackbits(v.view(np.uint8).reshape(len(v), 4), axis=1)  # noqa: E731
    assert np.all(np.abs(bits(x).mean(0) - 0.5) < 6 * 0.5 / np.sqrt(n))
    for y in (MA.state_hash(range(1, n + 1), 3, 17), MA.state_hash(range(n), 3, 18), MA.state_hash(range(n), 4, 17), MA.state_hash(range(256, n + 256), 3, 17)):
        assert np.all(np.abs(bits(x ^ y).mean(0) - 0.5) < 0.05)


def test_float8_grids_are_the_formats():
    import torch

    from oracle import many_adapters as MA

    e4 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    e5 = torch.arange(124, dtype=torch.uint8).view(torch.float8_e5m2).float().numpy()
    assert np.array_equal(MA.E4M3, e4) and np.array_equal(MA.E5M2, e5)


def test_pool_layer_refuses_planes_of_another_size():
    """The planes of T hold 3 M r elements; smaller ones are refused before any launch."""
    import types

    import torch

    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    pool = bd.AdapterPool(z(2, 8, 64), z(2, 16, 8), z(2, dt=torch.float32))
    q = types.SimpleNamespace(rows=16, cols=64, codes=z(16, 32, dt=torch.uint8))
    groups = (z(5, dt=torch.int32), z(3, dt=torch.int32))
    for planes in (z(2, 5, 8), z(3, 5, 8, dt=torch.float32), z(3, 8, 5).transpose(1, 2)):
        with pytest.raises(AssertionError):
            bd.linear_fwd_pool(q, pool, groups, z(5, 64), t_out=planes)
        with pytest.raises(AssertionError):
            bd.linear_bwd_pool(q, pool, groups, z(5, 64), z(5, 16), planes)


def test_the_stride_of_a_single_row_is_its_length():
    """One token may be a row of a tensor of any width: there is no next row."""
    import torch

    wide = torch.zeros(5, 100)
    assert bd._row_stride(wide[:, :64]) == 100 and bd._row_stride(wide[3:4, :64]) == 64
    assert bd._row_stride(wide[3:3, :64]) == 64 and bd._row_stride(wide.t()[:1, :1]) == 1
