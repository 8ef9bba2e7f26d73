"""The argument checks of the 4-bit and the few-token entry points, on the host:
every refusal comes before any device is touched, and empty calls succeed
without one."""
import ctypes

import numpy as np
import pytest
import torch

import w4_reference as ref

FAKE = 0x7F0000000000  # aligned, never dereferenced
MB = 1 << 20


def test_reference_packing():
    rng = np.random.default_rng(0)
    q = rng.integers(0, 16, (2, 21, 5))
    words = ref.pack(q)
    assert tuple(words.shape) == (2, 3, 5) and np.array_equal(ref.unpack(words, 21), q)
    assert int(ref.pack(np.array([[1], [2], [3]]))[0, 0]) == 0x321


QUANT = dict(matrices=1, K=64, N=16, group=32, B=FAKE, codes=FAKE + MB, scales=FAKE + 2 * MB, zeros=FAKE + 3 * MB)
BAD = [(dict(matrices=-1), 1), (dict(K=-1), 1), (dict(N=-1), 1), (dict(group=0), 1), (dict(group=16), 1), (dict(group=48), 1),
       (dict(group=2 ** 31), 1), (dict(matrices=2 ** 31), 2), (dict(matrices=2 ** 22, K=2 ** 21, N=2 ** 21), 2), (dict(K=2 ** 22), 2), (dict(N=2 ** 22), 2), (dict(B=0), 1),
       (dict(codes=0), 1), (dict(scales=0), 1), (dict(B=FAKE + 1), 1), (dict(codes=FAKE + MB + 2), 1),
       (dict(scales=FAKE + 2 * MB + 1), 1), (dict(codes=FAKE + 2044), 1), (dict(scales=FAKE + 2046), 1),
       (dict(zeros=FAKE + 2047), 1),
       (dict(matrices=0, B=0, codes=0, scales=0), 0), (dict(K=0, B=0, codes=0, scales=0, zeros=0), 0), (dict(N=0), 0)]


@pytest.mark.parametrize("change,status", BAD + [(dict(scales=FAKE + MB + 508), 1), (dict(zeros=FAKE + MB + 511), 1),
                                                 (dict(zeros=FAKE + 2 * MB + 63), 1)])
def test_quantize_refusals(native, change, status):
    a = {**QUANT, **change}
    assert native.quantize_w4(a["matrices"], a["K"], a["N"], a["group"], a["B"], a["codes"], a["scales"], a["zeros"], 0) == status


@pytest.mark.parametrize("change,status", BAD)
def test_dequantize_refusals(native, change, status):
    a = {**QUANT, **change}
    assert native.dequantize_w4(a["matrices"], a["K"], a["N"], a["group"], a["codes"], a["scales"], a["zeros"], a["B"], 0) == status


GEMM = dict(M=4, N=16, K=64, A=FAKE, group=32, codes=FAKE + MB, scales=FAKE + 2 * MB, zeros=FAKE + 3 * MB, bias=FAKE + 4 * MB,
            C=FAKE + 5 * MB, alpha=1.0, activation=0, workspace=FAKE + 6 * MB, workspace_bytes=4096)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=-1), 1), (dict(group=33), 1), (dict(M=2 ** 31), 2), (dict(N=2 ** 22), 2),
    (dict(K=2 ** 22), 2), (dict(A=0), 1), (dict(codes=0), 1), (dict(scales=0), 1), (dict(C=0), 1), (dict(A=FAKE + 1), 1),
    (dict(codes=FAKE + MB + 1), 1), (dict(scales=FAKE + 2 * MB + 1), 1), (dict(bias=FAKE + 4 * MB + 1), 1),
    (dict(C=FAKE + 5 * MB + 1), 1), (dict(workspace=FAKE + 6 * MB + 8), 1), (dict(workspace_bytes=-1), 1),
    (dict(alpha=float("inf")), 1), (dict(alpha=float("nan")), 1), (dict(activation=3), 1), (dict(activation=-1), 1),
    (dict(C=FAKE + 510), 1), (dict(C=FAKE + MB + 508), 1), (dict(C=FAKE + 2 * MB + 62), 1), (dict(C=FAKE + 3 * MB + 30), 1),
    (dict(C=FAKE + 4 * MB + 30), 1), (dict(C=FAKE + 6 * MB + 4094), 1), (dict(workspace=FAKE - 4080), 1),
    (dict(workspace=FAKE + MB), 1), (dict(workspace=FAKE + 3 * MB - 4080), 1),
    (dict(M=0, A=0, C=0), 0), (dict(N=0, codes=0, scales=0, C=0), 0),
])
def test_product_refusals(native, change, status):
    assert native.gemm_w4_scale_bias_act(*{**GEMM, **change}.values(), 0) == status


def test_workspace_sizes(native):
    assert native.w4_workspace_bytes(0, 5, 5) == 0
    assert native.w4_workspace_bytes(1, 4096, 4096) > 512
    for bad in ((-1, 4, 4), (4, 2 ** 22, 4), (4, 4, 2 ** 22), (2 ** 31, 4, 4)):
        with pytest.raises(native.GsrError):
            native.w4_workspace_bytes(*bad)
    assert native.expert_few_workspace_bytes(1, 2, 8, 11008, 4096) > 512
    for bad in ((-1, 2, 8, 4, 4), (65, 1, 8, 4, 4), (64, 17, 8, 4, 4), (1, 1025, 8, 4, 4), (4, 2, 1025, 4, 4),
                (4, 2, 8, 2 ** 22, 4), (4, 2, 8, 4, 2 ** 22)):
        with pytest.raises(native.GsrError):
            native.expert_few_workspace_bytes(*bad)


def few(native, tokens=4, k=2, experts=8, H=64, F=32, O=16, x=FAKE, ids=FAKE + MB, id_bytes=4, weights=FAKE + 2 * MB,
        up=(FAKE + 3 * MB, 0, 0, 0, 0), gate=None, down=(FAKE + 5 * MB, 0, 0, 0, 0), activation=1, out=FAKE + 7 * MB,
        ws=FAKE + 8 * MB, wsb=MB):
    def struct(t):
        return None if t is None else native.GsrWeights(*[v or None for v in t[:4]], t[4])

    return native.expert_mlp_few(tokens, k, experts, H, F, O, x, ids, id_bytes, weights, struct(up), struct(gate),
                                 struct(down), activation, out, ws, wsb, 0)


W4UP = (FAKE + 3 * MB, FAKE + 4 * MB, 0, 0, 32)
W4DOWN = (FAKE + 5 * MB, FAKE + 6 * MB, 0, 0, 64)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), 1), (dict(k=-1), 1), (dict(experts=-1), 1), (dict(H=-1), 1), (dict(F=-1), 1), (dict(O=-1), 1),
    (dict(id_bytes=2), 1), (dict(activation=4), 1), (dict(activation=-1), 1), (dict(wsb=-1), 1), (dict(wsb=512), 1),
    (dict(tokens=65), 2), (dict(k=257), 2), (dict(experts=1025), 2), (dict(H=2 ** 22), 2), (dict(F=2 ** 22), 2),
    (dict(O=2 ** 22), 2), (dict(k=2 ** 62), 2), (dict(k=256, F=2 ** 19), 2), (dict(x=0), 1), (dict(ids=0), 1), (dict(out=0), 1), (dict(ws=0), 1),
    (dict(up=(0, 0, 0, 0, 0)), 1), (dict(down=(0, 0, 0, 0, 0)), 1), (dict(gate=(0, 0, 0, 0, 0)), 1),
    (dict(x=FAKE + 1), 1), (dict(ids=FAKE + MB + 2), 1), (dict(ids=FAKE + MB + 4, id_bytes=8), 1),
    (dict(weights=FAKE + 2 * MB + 2), 1), (dict(out=FAKE + 7 * MB + 1), 1), (dict(ws=FAKE + 8 * MB + 8), 1),
    (dict(up=(FAKE + 3 * MB + 1, 0, 0, 0, 0)), 1), (dict(up=(FAKE + 3 * MB, 0, 0, FAKE + 1, 0)), 1),
    (dict(up=(FAKE + 3 * MB, FAKE, 0, 0, 0)), 1),                      # scales of fp16 weights
    (dict(up=W4UP), 1), (dict(down=W4DOWN), 1),                        # one of the two in 4 bits
    (dict(up=W4UP, down=W4DOWN, gate=(FAKE + 9 * MB, FAKE + 10 * MB, 0, 0, 64)), 1),  # gate of another group
    (dict(up=W4UP[:4] + (40,), down=W4DOWN), 1), (dict(up=(FAKE + 3 * MB, 0, 0, 0, 32), down=W4DOWN), 1),
    (dict(up=(FAKE + 3 * MB + 2,) + W4UP[1:], down=W4DOWN), 1),
    (dict(out=FAKE + 510), 1), (dict(out=FAKE + MB + 30), 1), (dict(out=FAKE + 2 * MB), 1), (dict(out=FAKE + 3 * MB + 64), 1),
    (dict(out=FAKE + 5 * MB - 126), 1), (dict(out=FAKE + 8 * MB - 2), 1), (dict(ws=FAKE + 6 * MB + 16), 1),
    (dict(ws=FAKE), 1),
    (dict(tokens=0, x=0, ids=0, weights=0, out=0), 0), (dict(O=0, down=(0, 0, 0, 0, 0), out=0), 0),
])
def test_few_refusals(native, change, status):
    assert few(native, **change) == status


def test_few_without_matrices(native):
    assert native.lib().gsr_expert_mlp_few(1, 1, 1, 1, 1, 1, FAKE, FAKE, 4, None, None, None, None, 0, FAKE, FAKE, 1, None) == 1


def test_python_refusals():
    import tiled_dense_gemm_scale_amd as gsr

    h, i32 = torch.zeros(64, 16, dtype=torch.float16), torch.zeros(8, 16, dtype=torch.int32)
    s = torch.zeros(2, 16, dtype=torch.float16)
    with pytest.raises(TypeError):
        gsr.quantize_w4(h.float())
    with pytest.raises(ValueError, match="shape"):
        gsr.quantize_w4(h[0])
    with pytest.raises(ValueError, match="device"):
        gsr.quantize_w4(h)
    with pytest.raises(TypeError, match="W4"):
        gsr.dequantize_w4(h)
    with pytest.raises(ValueError, match="device"):
        gsr.dequantize_w4(gsr.W4(i32, s, None, 64, 32))
    with pytest.raises(ValueError, match="group"):
        gsr.dequantize_w4(gsr.W4(i32, s, None, 64, 33))
    with pytest.raises(ValueError, match="device"):
        gsr.gemm_w4(h, gsr.W4(i32, s, None, 64, 32))
    with pytest.raises(ValueError, match="device"):
        gsr.expert_mlp_few(h, i32, None, h, h, torch.zeros(1, dtype=torch.uint8))


def test_bound_of_h():
    """h as two halves, hi + lo / 2048, is within 2^-22 of itself or 2^-35, and hi is
    zero for zeros alone: by the same steps in binary32 and binary16."""
    rng = np.random.default_rng(0)
    v = (2.0 ** rng.uniform(-149, 15.99, 400000) * rng.choice([-1.0, 1.0], 400000)).astype(np.float32)
    edges = np.float32(2.0) ** np.arange(-149, 16, dtype=np.float32)
    v = np.concatenate([v, edges, np.nextafter(edges, np.float32(0)), -np.nextafter(edges, np.float32(1e9)), [np.float32(65519.99)]])
    hi = v.astype(np.float16)
    lost = (hi == 0) & (v != 0)
    hi[lost] = np.copysign(np.float16(2.0 ** -24), v[lost])
    lo = ((v - hi.astype(np.float32)) * np.float32(2048)).astype(np.float16)
    assert np.isfinite(hi).all() and np.isfinite(lo).all() and (np.sign(hi) == np.sign(v)).all()
    v = v.astype(np.float64)
    assert (np.abs(hi.astype(np.float64) + lo.astype(np.float64) / 2048 - v) <= np.maximum(np.abs(v) * 2.0 ** -22, 2.0 ** -35)).all()
