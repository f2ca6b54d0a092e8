"""Expert ids of wider types than the kernels': those that 32 bits cannot hold are no expert's."""
import pytest
import torch

import bit_rotated_weight_b200 as tq

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
FAR = [2 ** 32 + 3, -(2 ** 32), 2 ** 32, 2 ** 31, -(2 ** 63), 2 ** 63 - 1, 2 ** 40 + 1, 4, -1]


def test_ids_that_do_not_fit_stay_outside():
    got = tq._ids32(torch.tensor(FAR + [0, 1, 2, 3]), 4)
    assert got.dtype == torch.int32
    assert all(not 0 <= i < 4 for i in got[:len(FAR)].tolist()) and got[len(FAR):].tolist() == [0, 1, 2, 3]
    far = tq._ids32(torch.tensor([2 ** 64 - 1, 2 ** 63, 2 ** 32 + 1, 2], dtype=torch.uint64), 4).tolist()
    assert far[3] == 2 and all(not 0 <= i < 4 for i in far[:3])
    for dtype in (torch.int8, torch.uint8, torch.int16, torch.int32):
        assert tq._ids32(torch.tensor([3, 0], dtype=dtype), 4).tolist() == [3, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("m", [len(FAR), 200])
def test_moe_skips_and_flags_them(m):
    g = torch.Generator().manual_seed(m)
    up = tq.tq4_1s_int8_quantize(torch.randn(4, 64, 96, generator=g).to(DEV))
    down = tq.tq4_1s_int8_quantize(torch.randn(4, 96, 64, generator=g).to(DEV))
    pu = tq.tq4_1s_quantize(torch.randn(4, 64, 96, generator=g).to(DEV), seed=1)
    pd = tq.tq4_1s_quantize(torch.randn(4, 96, 64, generator=g).to(DEV), seed=2)
    x = torch.randn(m, 96, generator=g).to(torch.bfloat16).to(DEV)
    tw = torch.rand(m, 2, generator=g).to(DEV)
    wide = torch.randint(0, 4, (m, 2), generator=g)
    wide[:len(FAR), 1] = torch.tensor(FAR)
    narrow = wide.clone()
    narrow[:len(FAR), 1] = -1
    tq.tq4_1s_get_status()
    for moe, u, d in ((tq.tq4_1s_moe_int8, up, down), (tq.tq4_1s_moe, pu, pd)):
        want = moe(x, narrow.to(torch.int32).to(DEV), tw, u, d)
        assert tq.tq4_1s_get_status() == tq.TQ_DEV_BAD_ROUTING
        assert torch.equal(moe(x, wide.to(DEV), tw, u, d), want)
        assert tq.tq4_1s_get_status() == tq.TQ_DEV_BAD_ROUTING
    a, b = tq.tq4_1s_moe_route(wide.to(DEV), 4), tq.tq4_1s_moe_route(narrow.to(torch.int32).to(DEV), 4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1][:int(a[0][-1])], b[1][:int(b[0][-1])])
