"""4-bit products, the expert step and quantisation at the ends of their ranges."""
import pytest
import torch

import tokens_ref as ref
from routed_expert_ffn_top_gb300 import moe

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def test_product_of_rows_past_2_gb():
    """fp32 rows of more than 2^31 bytes: their columns lie past a tensor store's coordinates.
    Channels of zeros but for three windows, whose sums are exact."""
    R, K, N = 33, 32, 2 ** 29 + 1024
    if torch.cuda.mem_get_info()[0] < 110 * 2 ** 30:
        pytest.skip("needs 110 GB of device memory")
    windows = [(0, 256), (2 ** 29 - 128, 2 ** 29 + 128), (N - 256, N)]
    g = gen(1)
    xc = torch.randint(0, 256, (R, K // 2), generator=g, dtype=torch.uint8)
    xs = torch.full((R, 16), 127, dtype=torch.uint8)
    wc = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.full((N, 16), 127, dtype=torch.uint8, device="cuda")
    part = {}
    for lo, hi in windows:
        c = torch.randint(0, 256, (hi - lo, K // 2), generator=g, dtype=torch.uint8)
        wc[lo:hi] = c.cuda()
        part[lo] = ref.values(xc, xs[:, :1]) @ ref.values(c, torch.full((hi - lo, 1), 127, dtype=torch.uint8)).T
    y = torch.full((R, N), float("nan"), device="cuda")
    work = torch.zeros(256, dtype=torch.uint8, device="cuda")
    moe.moe_microscale_product(xc.cuda(), xs.cuda(), wc, ws, out=y, workspace=work)
    assert moe.moe_read_device_status(work) == 0
    for lo, hi in windows:
        assert torch.equal(y[:, lo:hi].cpu().double(), part[lo])
    for r in (0, R - 1):
        for lo, hi in ((256, 2 ** 29 - 128), (2 ** 29 + 128, N - 256)):
            assert int(torch.count_nonzero(y[r, lo:hi])) == 0  # a NaN counts
    del y, wc, ws
    torch.cuda.empty_cache()
