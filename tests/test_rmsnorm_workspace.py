"""The workspace of the norm's backward pass stays small where rows are long (no GPU needed)."""
import pytest

from test_sequence_layers_ttt_amd import ttt


@pytest.mark.parametrize("io", [ttt.DTYPE_F32, ttt.DTYPE_BF16])
@pytest.mark.parametrize("rows,D", [(1024, 1 << 22), (5000, 1 << 20), (3, 1 << 26), (100000, 20000), (1, 70001)])
def test_long_rows(rows, D, io):
    """A rate for every row, and planes of dweight of 2^18 values together, or one."""
    need = ttt.rmsnorm_bwd_workspace_bytes(rows, D, io)
    assert 4 * (rows + D) <= need <= 4 * rows + 256 + 4 * max(D, 1 << 18)
