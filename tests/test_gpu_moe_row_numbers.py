"""The expert sort into the largest buffer there is: two pairs of one expert, padded to 2^31 - 1
rows (8.6 GB of row numbers), where a padded count or a step past the last row would leave 32
bits."""
import pytest

from tests.gpu_util import note

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_sort_to_the_last_row():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_fp8_linear_amd as m
    multiple = 2 ** 31 - 1
    idx = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    assert m.fp8_moe_rows(2, 1, 1, multiple) == multiple
    source = torch.full((multiple,), -99, dtype=torch.int32, device="cuda")
    note("moe_sort of two pairs into 2^31 - 1 rows")
    slot, _, counts, offsets = m.fp8_moe_sort(idx, 1, multiple, source=source)
    torch.cuda.synchronize()
    assert slot.flatten().tolist() == [0, 1] and counts.tolist() == [2]
    assert offsets.tolist() == [0, multiple] and source[:2].tolist() == [0, 1]
    assert all(bool((part == -1).all()) for part in source[2:].split(1 << 28))
