"""The gradient's workspace: a row of partial sums for each that is written, however long the rows are."""
import precision_tensor_core_gb300 as ptc


def test_long_rows_ask_for_what_they_use():
    """Rows of over 16384 elements have eight CTAs per SM of 152 in all, of 2048 columns each: 1216 pieces at most, or one
    set of partial sums."""
    import __graft_entry__
    __graft_entry__.build()
    f = ptc.ptc_rms_norm_backward_workspace
    for rows in (1, 3, 64, 512, 8192):
        for cols in (16385, 17001, 40000, 1 << 20, 1 << 24, 1 << 30):
            stats = rows * 8 + 16
            assert f(rows, cols) <= max(1216 * 2048 + cols, cols) * 4 + stats
            assert f(rows, cols) >= min(rows, max(1, 1216 // -(-cols // 2048))) * cols * 4 + rows * 8
    assert f(512, 16384) == 512 * 16384 * 4
