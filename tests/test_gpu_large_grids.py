"""GPU tests of products with more rows than one grid dimension holds threads:
they run on a tile whose launch fits, or are refused, never cut short."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def gsr(native):
    import tiled_dense_gemm_scale_amd as g

    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    return g


def grouped_identity(gsr, P, config_id=-1):
    """P rows of 8 values through a single group's identity; c equals a."""
    K = 8
    a = torch.empty(P, K, dtype=torch.float16, device=DEV).random_(-9, 9)
    b = torch.eye(K, dtype=torch.float16, device=DEV)[None].contiguous()
    offsets = torch.tensor([0, P], dtype=torch.int32, device=DEV)
    c = torch.full((P, K), 9.5, dtype=torch.float16, device=DEV)
    print(f"[gpu] grouped {P} rows config={config_id}", flush=True)
    try:
        gsr.gemm_grouped(a, b, offsets, activation="none", c=c, config_id=config_id)
        for lo in range(0, P, 1 << 28):
            assert torch.equal(c[lo:lo + (1 << 28)], a[lo:lo + (1 << 28)]), lo
    finally:
        del a, c
        torch.cuda.empty_cache()


def test_grouped_rows_past_a_grid(gsr):
    """2^29 rows: 2^32 threads with the 64 x 64 tile."""
    grouped_identity(gsr, 2 ** 29)
    with pytest.raises(gsr.GsrError) as e:
        grouped_identity(gsr, 2 ** 29, config_id=21)
    assert e.value.status == 2


def test_dense_rows_past_a_grid(gsr, native):
    """The element-wise 64 x 64 tile of 2^30 - 2 rows of one value: 2^24 tiles of
    256 threads."""
    M = 2 ** 30 - 2
    a = torch.empty(M, 1, dtype=torch.float16, device=DEV).random_(0, 9)
    b, c = torch.ones(1, 1, dtype=torch.float16, device=DEV), torch.full((M, 1), 9.5, dtype=torch.float16, device=DEV)
    for config in (21, 28):
        print(f"[gpu] dense {M} rows config={config}", flush=True)
        st = native.gemm_scale_bias_act(M, 1, 1, a.data_ptr(), b.data_ptr(), 0, c.data_ptr(), 1.0, 2, 0, config)
        torch.cuda.synchronize()
        assert st == 2 or (st == 0 and torch.equal(a, c))


def test_grouped_of_the_largest_count(gsr):
    """2^31 - 1 rows in one group: its tiles' count passes no 2^31 on the way."""
    grouped_identity(gsr, 2 ** 31 - 1)
