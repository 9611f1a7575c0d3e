"""CPU: what the low-rank adapter and checkpoint calls refuse, and the
reference's own pins. Nothing here reaches a GPU."""
import ctypes
import os

import numpy as np
import pytest
import torch

import lora_reference as R
from post_weight_quantization_26_amd import build_lib

FAKE = ctypes.c_void_p(0x10000)       # aligned, never dereferenced: validation fails first
MIS = ctypes.c_void_p(0x10008)        # not 16-byte aligned
ODD = ctypes.c_void_p(0x10002)        # not 4-byte aligned
BIG = 1 << 42


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(build_lib.LIB_PATH):
        build_lib.build()
    from post_weight_quantization_26_amd import _lib
    _lib.lib()
    return _lib


def common(L):
    return dict(dt=L.AWQ_BF16, T=40, N=264, K=384, qw=FAKE, qz=FAKE, sc=FAKE, g=128, A=FAKE,
                B=FAKE, c=FAKE, ids=FAKE, n=3, r=16, ws=FAKE, wsb=BIG)


def forward(L, **k):
    a = dict(common(L), X=FAKE, Y=FAKE, H=FAKE, x8=FAKE, xs=FAKE)
    a.update(k)
    return L.lib().awq_w4a16_lora_matmul(
        a["X"], a["dt"], a["T"], a["N"], a["K"], a["qw"], a["qz"], a["sc"], a["g"], a["A"], a["B"],
        a["c"], a["ids"], a["n"], a["r"], a["Y"], a["H"], a["x8"], a["xs"], a["ws"], a["wsb"],
        None)


def backward(L, **k):
    a = dict(common(L), dY=FAKE, X=FAKE, xs=FAKE, H=FAKE, dX=FAKE, dA=FAKE, dB=FAKE)
    a.update(k)
    return L.lib().awq_w4a16_lora_backward(
        a["dY"], a["X"], a["xs"], a["H"], a["dt"], a["T"], a["N"], a["K"], a["qw"], a["qz"],
        a["sc"], a["g"], a["A"], a["B"], a["c"], a["ids"], a["n"], a["r"], a["dX"], a["dA"],
        a["dB"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("call,name", [(forward, "w4a16_lora_matmul"),
                                       (backward, "w4a16_lora_backward")])
def test_refusals(L, call, name):
    INV, UNS, WS = L.AWQ_E_INVALID, L.AWQ_E_UNSUPPORTED, L.AWQ_E_WORKSPACE
    for k in ("qw", "qz", "sc", "A", "B", "c", "ids"):
        assert call(L, **{k: None}) == INV
        assert name in L.last_error()
        assert call(L, **{k: ODD}) == INV
    for k in ("qw", "qz", "sc", "A", "B"):
        assert call(L, **{k: MIS}) == INV
    assert call(L, dt=L.AWQ_F32) == UNS and call(L, dt=9) == INV
    for k in ("T", "N", "K", "n", "r"):
        assert call(L, **{k: 0}) == INV and call(L, **{k: -8}) == INV
    for k in ("T", "N", "K"):
        assert call(L, **{k: 1 << 31}) == INV
    assert call(L, N=260) == INV and call(L, K=200) == INV
    assert call(L, r=12) == UNS and call(L, r=136) == UNS
    assert call(L, n=4097) == UNS
    assert call(L, g=16) == UNS
    assert call(L, K=1 << 22) == UNS                       # 512·K reaches 2^31
    assert call(L, N=1 << 20, K=1 << 21) == UNS            # more than 2^34 weights
    assert call(L, T=(1 << 31) - 1, N=1 << 20) == UNS      # more work-items than a launch has
    assert call(L, ws=None) == WS and call(L, ws=MIS) == WS and call(L, wsb=16) == WS
    assert name in L.last_error()


def test_forward_refusals(L):
    INV = L.AWQ_E_INVALID
    assert forward(L, X=None) == INV and forward(L, Y=None) == INV
    assert forward(L, x8=None) == INV and forward(L, xs=None) == INV    # both or neither
    for k in ("X", "Y", "H", "x8"):
        assert forward(L, **{k: MIS}) == INV
    assert forward(L, xs=ODD) == INV


def test_backward_refusals(L):
    INV = L.AWQ_E_INVALID
    for k in ("dY", "X", "H", "dA", "dB"):
        assert backward(L, **{k: None}) == INV
        assert backward(L, **{k: MIS}) == INV
    assert backward(L, dX=MIS) == INV and backward(L, xs=ODD) == INV
    assert backward(L, N=1 << 22, K=128) == L.AWQ_E_UNSUPPORTED    # 512·N reaches 2^31


def test_workspace_sizes(L):
    for f in (L.lib().awq_w4a16_lora_workspace_bytes,
              L.lib().awq_w4a16_lora_backward_workspace_bytes):
        for T in (1, 16, 17, 64, 256, 4096):
            assert f(T, 4096, 4096, 4, 16, L.AWQ_BF16) > 0
        for bad in ((0, 8, 128, 1, 8, 1), (1, 12, 128, 1, 8, 1), (1, 8, 200, 1, 8, 1),
                    (1, 8, 128, 0, 8, 1), (1, 8, 128, 1, 12, 1), (1, 8, 128, 1, 136, 1),
                    (1, 8, 128, 4097, 8, 1), (1, 8, 128, 1, 8, 0), (1, 8, 128, 1, 8, 9)):
            assert f(*bad) == 0


def test_few_tokens_keep_no_layer_unless_offsets_need_one(L):
    """Up to 384 (gradient: 320) tokens no 16-bit layer is kept; a layer whose
    packed words pass 2^31 bytes in one run of k takes the other form."""
    f = L.lib().awq_w4a16_lora_workspace_bytes
    b = L.lib().awq_w4a16_lora_backward_workspace_bytes
    layer = 28672 * 8192 * 2
    assert f(384, 28672, 8192, 4, 16, L.AWQ_BF16) < layer <= f(385, 28672, 8192, 4, 16, L.AWQ_BF16)
    assert b(320, 28672, 8192, 1, 16, L.AWQ_BF16) < layer <= b(321, 28672, 8192, 1, 16, L.AWQ_BF16)
    for N, K, kept in ((1 << 25, 128, True), ((1 << 25) - 8, 128, False), (1 << 24, 512, False),
                       (1 << 23, 2048, True)):
        assert (f(17, N, K, 1, 8, L.AWQ_F16) >= N * K * 2) == kept


def test_checkpoint_refusals(L):
    lib = L.lib()
    INV, UNS = L.AWQ_E_INVALID, L.AWQ_E_UNSUPPORTED

    def pack(X=FAKE, dt=L.AWQ_BF16, T=4, K=256, c=FAKE, s=FAKE):
        return lib.awq_act_pack8(X, dt, T, K, c, s, None)

    def unpack(X=FAKE, dt=L.AWQ_BF16, T=4, K=256, c=FAKE, s=FAKE):
        return lib.awq_act_unpack8(c, s, dt, T, K, X, None)

    for f, name in ((pack, "act_pack8"), (unpack, "act_unpack8")):
        for k in ("X", "c", "s"):
            assert f(**{k: None}) == INV and f(**{k: ODD}) == INV
        assert name in L.last_error()
        assert f(X=MIS) == INV and f(c=MIS) == INV
        assert f(dt=9) == INV and f(T=0) == INV and f(K=0) == INV and f(K=200) == INV
        assert f(T=1 << 31) == INV
        assert f(T=1 << 28, K=256) == UNS                  # more than 2^34 elements


def test_python_refuses_tensors_off_the_gpu():
    from post_weight_quantization_26_amd import api
    with pytest.raises(ValueError, match="X must be a GPU tensor"):
        api.act_pack8(torch.zeros(2, 128))
    with pytest.raises(ValueError, match="X must be a GPU tensor"):
        api.w4a16_lora_matmul(torch.zeros(2, 128), *[None] * 7)
    with pytest.raises(ValueError, match="dY must be a GPU tensor"):
        api.w4a16_lora_backward(torch.zeros(2, 128), *[None] * 9)


def test_reference_checkpoint_pins():
    x = np.zeros((1, 128), np.float32)
    x[0, :5] = [127, 0.5, 1.5, -126.5, -2.5]      # step 1: ties go to the even code
    codes, steps = R.pack8(x)
    assert steps[0, 0] == 1 and codes[0, :5].tolist() == [127, 0, 2, -126, -2]
    codes, steps = R.pack8(np.zeros((2, 256), np.float32))
    assert not codes.any() and (steps == np.float32(2.0 ** -100) / np.float32(127)).all()
    x[0, 7] = np.inf
    codes, steps = R.pack8(x)
    assert not codes.any() and np.isnan(steps).all() and np.isnan(R.unpack8(codes, steps)).all()


def test_reference_gradient_by_brute_force():
    rng = np.random.default_rng(0)
    T, N, K, r, n = 5, 4, 6, 2, 2
    x, w, dy = (rng.standard_normal(s) for s in ((T, K), (N, K), (T, N)))
    A, B, c = rng.standard_normal((n, r, K)), rng.standard_normal((n, N, r)), rng.random(n)
    ids = np.array([0, 1, -1, 1, 7])
    loss = lambda x, A, B: (dy * R.forward(x, w, A, B, c, ids)[0]).sum()
    h = R.forward(x, w, A, B, c, ids)[1]
    dx, dA, dB = R.backward(dy, x, h, w, A, B, c, ids)[:3]
    for v, g, f in ((x, dx, lambda z: loss(z, A, B)), (A, dA, lambda z: loss(x, z, B)),
                    (B, dB, lambda z: loss(x, A, z))):
        num = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            d = np.zeros_like(v)
            d[i] = 1.0
            num[i] = (f(v + d) - f(v - d)) / 2
        assert np.allclose(num, g, atol=1e-12)
