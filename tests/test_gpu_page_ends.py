"""kda_page_release with the largest pools and tables that its 32-bit counts allow."""
import pytest
import torch

pytestmark = pytest.mark.gpu
I32 = torch.int32
MOST = 2 ** 31 - 1


def _i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


@pytest.mark.parametrize("pool", [MOST, MOST - 31, MOST - 300])
def test_the_largest_pools(cuda_lib, pool):
    """Pages at both ends of the pool given back, one of them still held by another row."""
    shares = torch.zeros(pool, dtype=I32, device="cuda")
    shares[pool - 1] = 1
    table = _i32([[pool - 1, 3, pool - 2, 0], [pool - 1, pool // 2, pool - 40, -1]])
    held, freed, n = cuda_lib.page_release(_i32([0, 8]), _i32([4, 3]), table, shares, page_size=8)
    assert held.tolist() == [0, 1] and n.item() == 5
    assert freed[:5].tolist() == sorted([3, pool - 2, 0, pool // 2, pool - 40]) and int((freed[5:] != -1).sum()) == 0
    assert not shares.any()
    held, freed, n = cuda_lib.page_release(_i32([0, 0]), held, table, shares, page_size=8)
    assert held.tolist() == [0, 0] and n.item() == 1 and freed[:2].tolist() == [pool - 1, -1] and not shares.any()
    assert cuda_lib.last_device_status() == cuda_lib.KDA_OK


@pytest.mark.parametrize("cols,held", [(MOST, MOST), (MOST, MOST - 200), (MOST - 255, MOST - 255)])
def test_the_widest_tables(cuda_lib, cols, held):
    """The last entries of a row given back."""
    table = torch.full((1, cols), -1, dtype=I32, device="cuda")
    ids = torch.randperm(1000, generator=torch.Generator().manual_seed(1))[:300].to(I32)
    table[0, held - 300:held] = ids.cuda()
    shares = torch.zeros(1000, dtype=I32, device="cuda")
    out, freed, n = cuda_lib.page_release(_i32([held - 300]), _i32([held]), table, shares, page_size=1)
    assert out.tolist() == [held - 300] and n.item() == 300 and torch.equal(freed[:300].cpu(), ids.sort().values) and not shares.any()
    assert (freed[300:] == -1).all() and cuda_lib.last_device_status() == cuda_lib.KDA_OK
