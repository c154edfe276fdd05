"""Rotary positions between parts of one buffer."""
import pytest
import torch

pytestmark = pytest.mark.gpu

qm = pytest.importorskip("quantized_matmul_amd")

DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 2, 37])
def test_from_one_part_of_the_rows_into_another(T, dtype):
    """x and out lie in the same rows and share no value: neighbours, either way round, and with a gap."""
    H, D = 3, 64
    freqs = qm.rotary_frequencies(D, device=DEV)
    positions = torch.arange(T, dtype=torch.int32, device=DEV) * 7
    for a, b, wide in ((0, H, 2 * H), (H, 0, 2 * H), (1, H + 2, 2 * H + 4), (H + 2, 1, 2 * H + 4)):
        rows = torch.randn((T, wide, D), device=DEV).to(dtype)
        before = rows.clone()
        want = qm.rotary(rows[:, a : a + H].contiguous(), positions, freqs)
        got = qm.rotary(rows[:, a : a + H], positions, freqs, out=rows[:, b : b + H])
        assert torch.equal(got, want)
        before[:, b : b + H] = want
        assert torch.equal(rows, before)


def test_parts_that_share_values_are_refused():
    H, D, T = 3, 64, 5
    freqs = qm.rotary_frequencies(D, device=DEV)
    positions = torch.arange(T, dtype=torch.int32, device=DEV)
    rows = torch.zeros((T, 3 * H, D), device=DEV, dtype=torch.bfloat16)
    for a, b in ((0, 1), (1, 0), (0, H - 1), (H, H + 1)):
        with pytest.raises(qm.QlinError):
            qm.rotary(rows[:, a : a + H], positions, freqs, out=rows[:, b : b + H])
    flat = rows.view(-1)
    for start in (D // 2, 8, H * D - 8):                              # in the middle of heads
        with pytest.raises(qm.QlinError):
            qm.rotary(rows[:, :H], positions, freqs, out=flat.as_strided((T, H, D), (3 * H * D, D, 1), start))
    with pytest.raises(qm.QlinError):                                 # rows that lie otherwise apart
        qm.rotary(rows[:, :H], positions, freqs, out=flat.as_strided((T, H, D), (2 * H * D, D, 1), H * D))
    with pytest.raises(qm.QlinError):                                 # the end of one row and the start of the next
        qm.rotary(rows[:4, :H], positions[:4], freqs, out=flat.as_strided((4, H, D), (3 * H * D, D, 1), (3 * H - 1) * D))
