"""Which of attention's kernels the shapes of attention_shapes run, from the workspace that
they ask for (no GPU)."""
import pytest

from attention_shapes import SHAPES, case_of

PAGE = 16


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("name", SHAPES)
def test_pieces(name, dim):
    from microscaling_block_scaled_amd import mx
    lens, Lq, heads, group, pieces = case_of(name, dim)
    rows = Lq * group
    most = (-(-max(lens) // PAGE) + 1) * PAGE  # as a table with a page to spare holds
    need = mx.lib.mx_attention_workspace(len(lens), Lq, heads * group, heads, dim, most)
    per = len(lens) * heads * (rows if rows <= 16 else -(-rows // 16) * 16) * (dim + 2) * 4
    assert need % per == 0 and (need > per if pieces else need == 0)
    assert (rows > 16) == ("rows a wave" in name) and (rows > 64) == ("32 rows" in name)
    if name == "eight waves" and dim < 256:
        assert most > 256  # four waves would cut it
    if "join" in name:  # one wave a row, the last workgroup not full
        assert len(lens) * heads * rows >= 2048 and len(lens) * heads * rows % 4
    elif rows <= 16:
        assert len(lens) * heads * rows < 2048
