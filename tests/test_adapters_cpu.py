"""The argument checks of the product with low-rank adapters, on the host."""
import math

import pytest
import torch

FAKE = 0x7F0000000000  # aligned, never dereferenced
GB = 1 << 30


def call(native, **change):
    a = dict(M=8, N=16, K=16, A=FAKE, B=FAKE + GB, bias=FAKE + 2 * GB, C=FAKE + 3 * GB, adapters=3, rank=8,
             la=FAKE + 4 * GB, lb=FAKE + 5 * GB, ids=FAKE + 6 * GB, scales=FAKE + 7 * GB, alpha=1.0, act=0,
             ws=FAKE + 8 * GB, wsb=1 << 20, stream=0, config_id=-1, splits=0)
    a.update(change)
    return native.gemm_adapters_scale_bias_act(*a.values())


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), 1), (dict(N=-1), 1), (dict(K=-1), 1), (dict(adapters=-1), 1), (dict(rank=-1), 1),
    (dict(splits=-1), 1), (dict(splits=17), 1), (dict(wsb=-1), 1),
    (dict(M=2 ** 31), 2), (dict(rank=257), 2), (dict(adapters=2 ** 31), 2),
    (dict(M=2 ** 20, K=2 ** 10), 2), (dict(N=2 ** 20, K=2 ** 10), 2), (dict(M=2 ** 20, N=2 ** 10), 2),
    (dict(M=1, K=1, N=2 ** 23, rank=128), 2),       # one adapter's Lb of 2^31 bytes
    (dict(alpha=math.nan), 1), (dict(act=3), 1), (dict(config_id=-2), 6), (dict(config_id=16), 6),
    (dict(config_id=28, splits=2), 6),
    (dict(A=0), 1), (dict(B=0), 1), (dict(C=0), 1), (dict(la=0), 1), (dict(lb=0), 1), (dict(ids=0), 1), (dict(ws=0), 1),
    (dict(A=FAKE + 1), 1), (dict(bias=FAKE + 2 * GB + 1), 1), (dict(la=FAKE + 4 * GB + 1), 1),
    (dict(lb=FAKE + 5 * GB + 1), 1), (dict(ids=FAKE + 6 * GB + 2), 1), (dict(scales=FAKE + 7 * GB + 2), 1),
    (dict(ws=FAKE + 8 * GB + 8), 1),
    (dict(C=FAKE + 4 * GB + 3 * 8 * 16 * 2 - 2), 1),  # C over the last La
    (dict(C=FAKE + 5 * GB - 254), 1),                 # C (256 bytes) over the first Lb
    (dict(C=FAKE + 6 * GB), 1), (dict(C=FAKE + 7 * GB), 1), (dict(C=FAKE + 8 * GB + 64), 1),
    (dict(ws=FAKE + 6 * GB - 32), 1), (dict(ws=FAKE + 4 * GB), 1),
    (dict(M=0), 0), (dict(N=0), 0),
])
def test_refusals(native, change, status):
    assert call(native, **change) == status


def test_workspace_bytes(native):
    assert native.adapter_workspace_bytes(0, 8, 8, 8) == 0
    assert native.adapter_workspace_bytes(8, 8, 8, 0) == 0
    for shape in ((1, 4096, 11008, 64), (16, 11008, 4096, 16), (4097, 11008, 4096, 16), (3, 5, 7, 1), (2048, 64, 4096, 256)):
        need = native.adapter_workspace_bytes(*shape)
        M, N, K, R = shape
        assert need >= 512 + M * ((R + 15) // 16) * (64 + 4)  # counters, a record and a scale per row and 16 ranks
    for bad in ((-1, 8, 8, 8), (8, 8, 8, 257), (8, 8, 8, -1)):
        with pytest.raises(native.GsrError):
            native.adapter_workspace_bytes(*bad)


def test_python_refusals():
    import tiled_dense_gemm_scale_amd as gsr

    h = dict(dtype=torch.float16)
    a, b, la, lb = torch.zeros(4, 8, **h), torch.zeros(8, 6, **h), torch.zeros(2, 3, 8, **h), torch.zeros(2, 6, 3, **h)
    ids, ws = torch.zeros(4, dtype=torch.int32), torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(TypeError):
        gsr.gemm_adapters(a.float(), b, la, lb, ids, ws)
    with pytest.raises(ValueError, match="device"):
        gsr.gemm_adapters(a, b, la, lb, ids, ws)


def test_more_rows_than_a_launch_has_threads(native):
    """From 2^27 - 15 rows on the inner sums' launch would have 2^32 threads."""
    far = dict(N=1, K=1, A=FAKE, B=FAKE + GB, bias=0, C=FAKE + 2 * GB, ws=FAKE + 20 * GB, wsb=100 * GB, la=FAKE + 10 * GB,
               lb=FAKE + 11 * GB, ids=FAKE + 12 * GB, scales=0)
    for M in (2 ** 27 - 15, 2 ** 27, 2 ** 29):
        assert call(native, M=M, **far) == 2
        with pytest.raises(native.GsrError):
            native.adapter_workspace_bytes(M, 1, 1, 8)
    assert native.adapter_workspace_bytes(2 ** 27 - 16, 1, 1, 8) > 0
