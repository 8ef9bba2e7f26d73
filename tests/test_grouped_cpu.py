"""The grouped products' argument checks, on the host."""
import math

import pytest
import torch

FAKE = 0x7F0000000000  # aligned, never dereferenced
GB = 1 << 30


def call(native, **change):
    a = dict(P=8, N=16, K=16, groups=3, A=FAKE, a_rows=4, rows=FAKE + GB, B=FAKE + 2 * GB, bias=FAKE + 3 * GB,
             C=FAKE + 4 * GB, offsets=FAKE + 5 * GB, alpha=1.0, act=0, stream=0, config_id=-1)
    a.update(change)
    return native.gemm_grouped_scale_bias_act(*a.values())


@pytest.mark.parametrize("change,status", [
    (dict(P=-1), 1), (dict(N=-1), 1), (dict(K=-1), 1), (dict(groups=-1), 1), (dict(a_rows=-1), 1),
    (dict(P=2 ** 31), 2), (dict(N=2 ** 22), 2), (dict(K=2 ** 22), 2), (dict(groups=1025), 2),
    (dict(K=2 ** 16, N=2 ** 14), 2),                 # one group's B of 2^31 bytes
    (dict(a_rows=2 ** 20, K=2 ** 10), 2),            # A behind rows of 2^31 bytes
    (dict(alpha=math.inf), 1), (dict(alpha=math.nan), 1), (dict(act=3), 1), (dict(act=-1), 1),
    (dict(config_id=-2), 6), (dict(config_id=16), 6), (dict(config_id=99), 6),
    (dict(A=0), 1), (dict(B=0), 1), (dict(C=0), 1), (dict(offsets=0), 1),
    (dict(A=FAKE + 1), 1), (dict(B=FAKE + 2 * GB + 1), 1), (dict(C=FAKE + 4 * GB + 1), 1),
    (dict(bias=FAKE + 3 * GB + 1), 1), (dict(rows=FAKE + GB + 2), 1), (dict(offsets=FAKE + 5 * GB + 1), 1),
    (dict(C=FAKE + 100), 1),                         # C inside A (4 x 16)
    (dict(C=FAKE + GB + 28), 1),                     # C over the last of rows
    (dict(C=FAKE + 2 * GB + 3 * 16 * 16 * 2 - 2), 1),  # C over the last group's B
    (dict(C=FAKE + 3 * GB + 94), 1),                 # C over the last bias
    (dict(C=FAKE + 5 * GB + 12), 1),                 # C over offsets
    (dict(rows=0, C=FAKE + 254), 1),                 # without rows A has P rows
    (dict(P=0, A=0, B=0, C=0, offsets=0), 0), (dict(N=0, B=0, C=0), 0), (dict(groups=0, B=0, offsets=0), 0),
])
def test_refusals(native, change, status):
    assert call(native, **change) == status


def test_python_refusals():
    import tiled_dense_gemm_scale_amd as gsr

    a, b = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(2, 8, 16, dtype=torch.float16)
    o = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        gsr.gemm_grouped(a.float(), b, o)
    with pytest.raises(ValueError, match="device"):
        gsr.gemm_grouped(a, b, o)


@pytest.mark.parametrize("change,status", [
    (dict(P=2 ** 29, config_id=21), 2), (dict(P=2 ** 28, config_id=22), 2), (dict(P=2 ** 30, config_id=31), 2),
    (dict(P=2 ** 31 - 1, K=1, N=1, config_id=28), 2),  # 2^24 tiles of 256 threads
])
def test_launches_of_too_many_threads(native, change, status):
    """2^32 threads and more, of which a launch would run a part."""
    far = dict(groups=1, a_rows=0, rows=0, N=8, K=8, C=FAKE + 100 * GB, B=FAKE + 200 * GB, bias=0, offsets=FAKE + 201 * GB)
    assert call(native, **{**far, **change}) == status
