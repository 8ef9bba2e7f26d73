"""The row entry points' argument checks, on the host: every refusal comes
before any device is touched, and empty calls succeed without one."""
import pytest
import torch

FAKE = 0x7F0000000000  # aligned, never dereferenced
MB = 1 << 20


def group(native, tokens=4, k=2, groups=8, ids=FAKE, id_bytes=4, offsets=FAKE + MB, rows=FAKE + 2 * MB,
          positions=FAKE + 3 * MB, ws=0, wsb=0):
    return native.group_rows(tokens, k, groups, ids, id_bytes, offsets, rows, positions, ws, wsb, 0)


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), 1), (dict(k=-1), 1), (dict(groups=0), 1), (dict(groups=-3), 1), (dict(id_bytes=2), 1),
    (dict(groups=1025), 2), (dict(tokens=2 ** 31), 2), (dict(tokens=2 ** 16, k=2 ** 16), 2),
    (dict(ids=0), 1), (dict(offsets=0), 1), (dict(rows=0), 1), (dict(positions=0), 1),
    (dict(ids=FAKE + 2), 1), (dict(ids=FAKE + 4, id_bytes=8), 1), (dict(offsets=FAKE + MB + 2), 1),
    (dict(rows=FAKE + 2 * MB + 1), 1), (dict(positions=FAKE + 3 * MB + 3), 1),
    (dict(rows=FAKE + 28), 1),                               # rows begins inside ids
    (dict(positions=FAKE + 2 * MB + 4), 1),                  # positions inside rows
    (dict(offsets=FAKE + 16), 1),                            # offsets inside ids
    (dict(wsb=-1), 1),
    (dict(tokens=8193, k=1), 1),                             # needs a workspace
    (dict(tokens=8193, k=1, ws=FAKE + 8 * MB, wsb=107), 1),  # 3 blocks x 9 counts x 4 bytes = 108
    (dict(tokens=8193, k=1, ws=FAKE + 8 * MB + 8, wsb=108), 1),
    (dict(tokens=8193, k=1, ws=FAKE, wsb=108), 1),           # the workspace over ids
])
def test_group_refusals(native, change, status):
    assert group(native, **change) == status


def test_group_workspace_bytes(native):
    assert native.group_workspace_bytes(0, 8) == 0
    assert native.group_workspace_bytes(8192, 1024) == 0
    assert native.group_workspace_bytes(8193, 8) == 5 * 9 * 4  # blocks of 2048 slots
    assert native.group_workspace_bytes(131072, 64) == 64 * 65 * 4
    # never more than 256 blocks
    assert native.group_workspace_bytes(2 ** 31 - 1, 1024) <= 256 * 1025 * 4
    for bad in ((-1, 8), (4, 0), (4, 1025)):
        with pytest.raises(native.GsrError):
            native.group_workspace_bytes(*bad)


@pytest.mark.parametrize("args,status", [
    ((-1, 4, 8, FAKE, FAKE + MB, FAKE + 2 * MB), 1), ((4, -1, 8, FAKE, FAKE + MB, FAKE + 2 * MB), 1),
    ((4, 4, -8, FAKE, FAKE + MB, FAKE + 2 * MB), 1), ((2 ** 31, 4, 8, FAKE, FAKE + MB, FAKE + 2 * MB), 2),
    ((4, 4, 2 ** 30, FAKE, FAKE + MB, FAKE + 2 * MB), 2),
    ((4, 4, 8, 0, FAKE + MB, FAKE + 2 * MB), 1), ((4, 4, 8, FAKE, 0, FAKE + 2 * MB), 1),
    ((4, 4, 8, FAKE, FAKE + MB, 0), 1), ((4, 4, 8, FAKE + 1, FAKE + MB, FAKE + 2 * MB), 1),
    ((4, 4, 8, FAKE, FAKE + MB + 2, FAKE + 2 * MB), 1), ((4, 4, 8, FAKE, FAKE + MB, FAKE + 2 * MB + 1), 1),
    ((4, 4, 8, FAKE, FAKE + MB, FAKE + 62), 1),        # out begins inside x
    ((4, 4, 8, FAKE, FAKE + MB + 16, FAKE + MB), 1),   # out over rows
    ((0, 4, 8, 0, 0, 0), 0), ((4, 4, 0, 0, 0, 0), 0),  # nothing to write
])
def test_gather_refusals(native, args, status):
    assert native.gather_rows(*args, 0) == status


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), 1), (dict(k=-1), 1), (dict(rows_in=-1), 1), (dict(width=-1), 1),
    (dict(tokens=2 ** 20, k=2 ** 12), 2), (dict(rows_in=2 ** 31), 2), (dict(width=2 ** 30), 2),
    (dict(y=0), 1), (dict(positions=0), 1), (dict(out=0), 1), (dict(y=FAKE + 1), 1), (dict(out=FAKE + 3 * MB + 1), 1),
    (dict(positions=FAKE + MB + 2), 1), (dict(weights=FAKE + 2 * MB + 2), 1),
    (dict(out=FAKE + 16), 1), (dict(out=FAKE + MB), 1), (dict(out=FAKE + 2 * MB), 1),
    (dict(tokens=0, y=0, positions=0, weights=0, out=0), 0), (dict(width=0, y=0, out=0), 0),
])
def test_combine_refusals(native, change, status):
    a = dict(tokens=4, k=2, rows_in=8, width=8, y=FAKE, positions=FAKE + MB, weights=FAKE + 2 * MB, out=FAKE + 3 * MB)
    a.update(change)
    assert native.combine_rows(*a.values(), 0) == status


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), 1), (dict(width=-1), 1), (dict(tokens=2 ** 20, k=2 ** 12), 2), (dict(width=2 ** 30), 2),
    (dict(weights=0), 1), (dict(dweights=0), 1),   # both or neither
    (dict(y=0), 1), (dict(dout=0), 1), (dict(positions=0), 1), (dict(rows=0), 1), (dict(dy=0), 1),
    (dict(dy=FAKE + 16), 1), (dict(dy=FAKE + MB), 1), (dict(dweights=FAKE + 5 * MB + 32), 1),
    (dict(dweights=FAKE + 2 * MB), 1), (dict(rows=FAKE + 4 * MB + 2), 1), (dict(dout=FAKE + 1), 1),
    (dict(tokens=0, rows_in=0, dout=0, y=0, positions=0, rows=0, dy=0), 0),
    (dict(weights=0, dweights=0, rows_in=0, y=0, rows=0, dy=0), 0),
])
def test_combine_backward_refusals(native, change, status):
    a = dict(tokens=4, k=2, rows_in=8, width=8, dout=FAKE, y=FAKE + MB, positions=FAKE + 2 * MB, weights=FAKE + 3 * MB,
             rows=FAKE + 4 * MB, dy=FAKE + 5 * MB, dweights=FAKE + 6 * MB)
    a.update(change)
    assert native.combine_rows_backward(*a.values(), 0) == status


def test_python_refusals():
    import tiled_dense_gemm_scale_amd as gsr

    i32, h = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(8, 16, dtype=torch.float16)
    with pytest.raises(TypeError):
        gsr.group_rows(i32.float(), 4)
    with pytest.raises(ValueError, match="shape"):
        gsr.group_rows(torch.zeros(2, 2, 2, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="device"):
        gsr.group_rows(i32, 4)
    with pytest.raises(TypeError):
        gsr.gather_rows(h.float(), i32.reshape(-1))
    with pytest.raises(ValueError, match="device"):
        gsr.gather_rows(h, i32.reshape(-1))
    with pytest.raises(ValueError, match="device"):
        gsr.combine_rows(h, i32)
    with pytest.raises(TypeError):
        gsr.combine_rows_backward(h.double(), h, i32, None, i32.reshape(-1))
