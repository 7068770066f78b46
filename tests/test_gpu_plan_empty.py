"""GPU tests of kv_slots and kv_slots_packed with lists of no entry: what there is no room for is reported
as at any other width."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(gkr, packed, lengths, first, width):
    t = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    table = torch.arange(3 * len(lengths), dtype=torch.int32, device=DEV).view(len(lengths), 3)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    f = gkr.kv_slots_packed if packed else gkr.kv_slots
    got = f(table, t(lengths), 4, width, first=t(first), err_flag=err)
    return got, int(err.item())


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("lengths,first,bad", [
    ([0, 5, 0], None, True), ([0, 0], None, False), ([3, 7], [3, 7], False), ([3, 7], [3, 6], True),
    ([0, -1], None, True), ([0, 0], [0, -2], True), ([1] * 5000, None, True), ([0] * 5000, None, False)])
def test_no_room(gkr, packed, lengths, first, bad):
    got, err = run(gkr, packed, lengths, first, 0)
    assert err == (gkr.ERR_INDEX if bad else 0)
    if packed:
        n = torch.tensor(lengths).clamp(min=0) - torch.tensor(first or [0] * len(lengths)).clamp(min=0)
        assert got[0].shape == (0,) and got[1].tolist() == [0, *n.clamp(min=0).cumsum(0).tolist()]
    else:
        assert got.shape == (len(lengths), 0)


def test_no_room_and_no_flag(gkr):
    lengths = torch.tensor([4, 5], dtype=torch.int32, device=DEV)
    table = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    assert gkr.kv_slots(table, lengths, 4, 0).shape == (2, 0)
    assert gkr.kv_slots(table[:0], lengths[:0], 4, 0).shape == (0, 0)
