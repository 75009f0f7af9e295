"""The 64-bit statement of the 4-bit operators against its own definitions (no GPU needed)."""
import torch

import w4a4_reference as ref


def test_nearest_takes_ties_to_even():
    v = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 100.0, 0.26], dtype=torch.float64)
    got = [ref.E2M1[i] for i in ref.nearest(v, ref.E2M1).tolist()]
    assert got == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0, 0.5]
    assert ref.E4M3[-1] == 448.0 and ref.E4M3[8] == 2.0 ** -6 and len(ref.E4M3) == 127
    mid = (ref.E4M3[40] + ref.E4M3[41]) / 2
    assert ref.nearest(torch.tensor([mid], dtype=torch.float64), ref.E4M3).item() == 40


def test_row_scale_is_the_smallest_power():
    x = torch.zeros(6, 16)
    for i, v in enumerate((2688.0, 2704.0, 1.3125, 0.0, 3.0e38, 1e-38)):
        x[i, 3] = v
    _, _, r = ref.quantize(x.bfloat16())
    top = x.bfloat16().double().abs().amax(1)
    assert r[3] == 1 and r[4] <= 2.0 ** 117 and r[5] == 2.0 ** -100
    for i in (0, 1, 2, 4):
        assert top[i] <= 2688 * r[i] and top[i] > 2688 * r[i] / 2


def test_values_of_representable_rows_come_back():
    g = torch.Generator().manual_seed(1)
    c = torch.tensor(ref.E2M1)[torch.randint(0, 8, (40, 64), generator=g)]
    c *= 1 - 2 * torch.randint(0, 2, (40, 64), generator=g)
    c[:, ::16] = 6.0  # each block's largest
    s = torch.tensor(ref.E4M3)[torch.randint(64, 120, (40, 4), generator=g)]
    s[:, 0] = 448.0   # the row's largest
    x = (c.view(40, 4, 16) * s[..., None]).view(40, 64) * 2.0 ** -7
    assert torch.equal(x, x.bfloat16().float())
    assert torch.equal(ref.values(x.bfloat16()), x.double())


def test_order_lists():
    ids = torch.tensor([[2, 0], [0, -1], [5, 2]], dtype=torch.int32)
    start, source, place = ref.order(ids, 3)
    assert start.tolist() == [0, 2, 2, 4]
    assert source.tolist() == [0, 1, 0, 2, -1, -1]
    assert place.tolist() == [[2, 0], [1, -1], [-1, 3]]
