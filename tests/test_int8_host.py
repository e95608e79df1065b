"""Refusals and size queries of the int8 layer and the group norm (CPU: every error is reported before any
CUDA call), and the binding's own checks of tensors."""
import pytest
import torch

from w4a4_rank_absorbed_b200 import build, svdq as C
from w4a4_rank_absorbed_b200.calib import calibrate_w8a8
from w4a4_rank_absorbed_b200.layer import GroupNorm, W8A8Linear

OK, INVAL, UNSUP, ALIGN = (C.SVDQ_OK, C.SVDQ_ERR_INVALID_ARG, C.SVDQ_ERR_UNSUPPORTED_SHAPE, C.SVDQ_ERR_MISALIGNED)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return C.load_library()


def _call(lib, name, defaults, **kw):
    a = dict(defaults)
    assert not set(kw) - set(a)
    a.update(kw)
    return getattr(lib, name)(*a.values(), None)


LINEAR = dict(Xq=16, sx=16, Wq=16, sw=16, bias=None, Y=16, y_type=0, ldy=96, M=3, N=96, K=64)
QUANT = dict(X=16, x_type=0, ldx=64, M=3, K=64, inv_s=16, Xq=16, sx=16)
FORWARD = dict(X=16, x_type=0, ldx=64, inv_s=16, Wq=16, sw=16, bias=None, Y=16, y_type=0, ldy=96, M=3, N=96, K=64,
               ws=16, wsb=1 << 20)
NORM = dict(X=16, type=0, ldx=64, B=2, S=3, C=64, G=4, gamma=16, beta=16, eps=1e-5, act=0, Y=16, ldy=64, ws=16,
            wsb=1 << 30)
NORMQ = dict(X=16, type=0, ldx=64, B=2, S=3, C=64, G=4, gamma=16, beta=16, eps=1e-5, act=0, inv_s=16, Xq=16, sx=16,
             ws=16, wsb=1 << 30)


@pytest.mark.parametrize("name,base,cases", [
    ("svdq_linear_i8", LINEAR, [
        (dict(K=72), UNSUP), (dict(K=1 << 17), UNSUP), (dict(K=0), INVAL), (dict(N=0), INVAL), (dict(M=-1), INVAL),
        (dict(M=1 << 31), UNSUP), (dict(M=(1 << 31) - 1023), UNSUP), (dict(N=1 << 31, ldy=1 << 31), UNSUP), (dict(Xq=None), INVAL), (dict(sx=None), INVAL),
        (dict(Wq=None), INVAL), (dict(sw=None), INVAL), (dict(Y=None), INVAL), (dict(y_type=3), INVAL),
        (dict(y_type=-1), INVAL), (dict(ldy=95), INVAL), (dict(Xq=8), ALIGN), (dict(Y=24), ALIGN), (dict(bias=8), ALIGN),
        (dict(sw=4), ALIGN), (dict(M=0, Xq=None, sx=None, Y=None), OK), (dict(M=0, K=72), UNSUP),
        (dict(ldy=(1 << 40) + 1), UNSUP)]),
    ("svdq_quantize_act_i8", QUANT, [
        (dict(K=24, ldx=24), UNSUP), (dict(ldx=63), INVAL), (dict(ldx=65), ALIGN), (dict(x_type=1, ldx=66), ALIGN),
        (dict(x_type=7), INVAL), (dict(X=None), INVAL), (dict(X=2), ALIGN), (dict(Xq=None), INVAL),
        (dict(sx=None), INVAL), (dict(inv_s=4), ALIGN), (dict(M=0, X=None, Xq=None, sx=None), OK), (dict(M=-1), INVAL)]),
    ("svdq_forward_i8", FORWARD, [
        (dict(K=72, ldx=72), UNSUP), (dict(ws=None), INVAL), (dict(wsb=3 * 64 + 3 * 4 - 1), INVAL), (dict(ws=8), ALIGN),
        (dict(X=None), INVAL), (dict(Wq=None), INVAL), (dict(y_type=5), INVAL), (dict(x_type=5), INVAL),
        (dict(ldx=60), INVAL), (dict(ldy=5), INVAL), (dict(M=0, X=None, Y=None, ws=None, wsb=0), OK)]),
    ("svdq_group_norm", NORM, [
        (dict(G=5), UNSUP), (dict(C=4104, ldx=4104, ldy=4104), UNSUP), (dict(G=0), INVAL), (dict(C=0), INVAL),
        (dict(B=-1), INVAL), (dict(S=-1), INVAL), (dict(B=1 << 16, S=1 << 16), UNSUP), (dict(B=1, S=(1 << 30) + 1), UNSUP), (dict(type=3), INVAL),
        (dict(act=3), INVAL), (dict(act=-1), INVAL), (dict(eps=-1.0), INVAL), (dict(eps=float("nan")), INVAL),
        (dict(eps=float("inf")), INVAL), (dict(X=None), INVAL), (dict(Y=None), INVAL), (dict(ldx=63), INVAL),
        (dict(ldy=63), INVAL), (dict(X=2), ALIGN), (dict(ws=None), INVAL), (dict(wsb=8), INVAL), (dict(ws=8), ALIGN),
        (dict(gamma=4), ALIGN), (dict(B=0, X=None, Y=None, ws=None), OK), (dict(S=0, X=None, Y=None, ws=None), OK),
        (dict(S=0, G=5), UNSUP)]),
    ("svdq_group_norm_quantize_i8", NORMQ, [
        (dict(C=72, ldx=72), UNSUP), (dict(Xq=None), INVAL), (dict(sx=None), INVAL), (dict(Xq=8), ALIGN),
        (dict(inv_s=4), ALIGN), (dict(wsb=8), INVAL), (dict(S=0, X=None, Xq=None, sx=None, ws=None), OK)]),
    ("svdq_pack_weight_i8", dict(W=16, K=64, N=3, Wq=16, sw=16), [
        (dict(K=8), UNSUP), (dict(N=0), INVAL), (dict(W=None), INVAL), (dict(W=4), ALIGN), (dict(Wq=8), ALIGN)]),
])
def test_refusals(lib, name, base, cases):
    for kw, want in cases:
        got = _call(lib, name, base, **kw)
        assert got == want, (name, kw, C.status_string(got), C.status_string(want))
    if not torch.cuda.is_available():
        assert _call(lib, name, base) in (C.SVDQ_ERR_CUDA, C.SVDQ_ERR_DEVICE)


def test_sizes(lib):
    assert C.svdq_forward_i8_workspace_bytes(7, 64) == 7 * 64 + 7 * 4
    assert C.svdq_forward_i8_workspace_bytes(0, 64) == 0
    assert C.svdq_forward_i8_workspace_bytes(7, 60) == 0
    assert C.svdq_group_norm_workspace_bytes(2, 100, 64, 4) > 0
    assert C.svdq_group_norm_workspace_bytes(2, 100, 64, 5) == 0
    assert C.svdq_group_norm_workspace_bytes(2, 100, 8192, 32) == 0


def test_rows_of_strided_tensors():
    """CPU tensors stand in (device index -1): the pitch the library is given, or the refusal."""
    t = torch.zeros(4, 6, 32, dtype=torch.bfloat16)
    assert C._rows(t, 24, 32, -1, "t")[1:] == (C.SVDQ_BF16, 32)
    assert C._rows(t[:, :, 8:24], 24, 16, -1, "t")[1:] == (C.SVDQ_BF16, 32)
    assert C._rows(t[:, ::2, :], 12, 32, -1, "t")[1:] == (C.SVDQ_BF16, 64)
    assert C._rows(t[:, :1, :], 4, 32, -1, "t")[1:] == (C.SVDQ_BF16, 6 * 32)
    assert C._rows(t[:1, :1, 3:5], 1, 2, -1, "t")[1:] == (C.SVDQ_BF16, 2)
    assert C._rows(torch.zeros(32, dtype=torch.float16), 1, 32, -1, "t")[1:] == (C.SVDQ_FP16, 32)
    assert C._rows(torch.zeros(0, 32), 0, 32, -1, "t")[1:] == (C.SVDQ_FP32, 32)
    for bad, rows, width in ((t[:, :4, :], 16, 32),              # two pitches
                             (t.transpose(1, 2), 128, 6),        # columns not contiguous
                             (t[0, :1].expand(6, 32), 6, 32),    # the same row again and again
                             (t[:, :1].expand(4, 3, 32), 12, 32), (t[:1].expand(4, 6, 32), 24, 32),
                             (t[:, :1, :1].expand(4, 3, 1), 12, 1), (t[:, :, :1].expand(4, 6, 5), 24, 5),
                             (t, 23, 32), (t, 24, 31)):
        with pytest.raises(ValueError):
            C._rows(bad, rows, width, -1, "t")
    with pytest.raises(TypeError):
        C._rows(torch.zeros(2, 2, dtype=torch.int8), 2, 2, -1, "t")


def test_vectors_are_checked():
    t = torch.zeros(8)
    assert C._vec(None, torch.float32, 8, -1, "t") == 0
    assert C._vec(t, torch.float32, 8, -1, "t") == t.data_ptr()
    for bad, kind in ((t[::2], ValueError), (t[:7], ValueError), (t.double(), TypeError)):
        with pytest.raises(kind):
            C._vec(bad, torch.float32, 4 if bad is not t[:7] and bad.numel() == 4 else 8, -1, "t")
    with pytest.raises(ValueError):
        C._vec(t, torch.float32, 8, 0, "t")                      # another device
    with pytest.raises(ValueError):
        C.svdq_linear_i8(t, t, t, t, None, t, 1, 1, 16)          # CPU tensors


def test_layer_arguments():
    with pytest.raises(ValueError):
        GroupNorm(3, 64, device="cpu")
    with pytest.raises(ValueError):
        GroupNorm(4, 64, act="relu", device="cpu")
    with pytest.raises(ValueError):
        GroupNorm(4, 64, weight=torch.ones(63), device="cpu")
    n = GroupNorm(4, 64, device="cpu")
    with pytest.raises(ValueError):
        n.forward(torch.zeros(2, 63))
    with pytest.raises(ValueError):
        n.forward(torch.zeros(64))
    with pytest.raises(ValueError):
        W8A8Linear.from_state_dict({"K": 16, "N": 4, "Wq": torch.zeros(4, 15, dtype=torch.int8), "sw": torch.zeros(4),
                                    "inv_s": None, "bias": None}, device="cpu")
    layer = W8A8Linear.from_state_dict({"K": 16, "N": 4, "Wq": torch.zeros(4, 16, dtype=torch.int8), "sw": torch.zeros(4),
                                        "inv_s": None, "bias": None}, device="cpu")
    for codes in (torch.zeros(2, 32, dtype=torch.int8), torch.zeros(32, dtype=torch.int8)):
        with pytest.raises(ValueError, match="Xq must be"):
            layer.gemm(codes, torch.zeros(2), torch.zeros(2, 4))


def test_calibration_smooths():
    g = torch.Generator().manual_seed(1)
    X, W = torch.randn(32, 48, generator=g), torch.randn(48, 24, generator=g)
    X[:, 7] *= 40
    W[3] = 0
    d = calibrate_w8a8(X, W, bias=torch.ones(24))
    assert (d.K, d.N) == (48, 24) and d.bias.dtype == torch.float32 and float(d.s[3]) == 1.0
    want = (X.double().abs().amax(0) / W.double().abs().amax(1)).sqrt()
    keep = torch.arange(48) != 3
    assert torch.allclose(d.s[keep], want[keep])
    assert torch.allclose((X.double() * d.inv_s) @ d.W_hat.double(), X.double() @ W.double(), rtol=1e-5, atol=1e-5)


def test_packed_calls_are_the_calls(lib):
    """svdq_call unpacks each entry point's arguments in their order: the refusal of one changed argument at a time
    is the entry point's own."""
    import struct
    for entry, name, base in ((C._quantize_act_i8, "svdq_quantize_act_i8", QUANT), (C._linear_i8, "svdq_linear_i8", LINEAR),
                              (C._forward_i8, "svdq_forward_i8", FORWARD), (C._group_norm, "svdq_group_norm", NORM),
                              (C._group_norm_quantize_i8, "svdq_group_norm_quantize_i8", NORMQ)):
        seen = set()
        for key, old in base.items():
            for new in (None, -1, 3, 8, 1 << 40):
                if key == "eps":
                    new = -1.0 if new is None else float(new)
                elif new is None and isinstance(old, int) and key[0].islower() and key not in ("ws", "sx", "sw", "inv_s",
                                                                                            "gamma", "beta"):
                    continue
                elif new is None and key in "MNKBSCG":
                    continue
                elif new in (-1, 1 << 40) and key not in ("M", "N", "K", "B", "S", "C", "G", "ldx", "ldy"):
                    continue
                args = dict(base, **{key: new})
                direct = _call(lib, name, base, **{key: new})
                if direct in (C.SVDQ_OK, C.SVDQ_ERR_CUDA, C.SVDQ_ERR_DEVICE):
                    continue                        # accepted: nothing to compare without a launch
                seen.add((key, direct))
                block = entry.pack(*[0 if v is None else v for v in args.values()], 0)
                assert lib.svdq_call(entry.index, block) == direct, (name, key, new)
        assert len(seen) >= 8
    assert lib.svdq_call(5, b"\0" * 200) == INVAL and lib.svdq_call(-1, b"\0" * 200) == INVAL
    assert lib.svdq_call(0, None) == INVAL
    block = struct.pack("<16q", *([0] * 16))
    assert lib.svdq_call(1, block) == INVAL
