"""Refusals of overlapping buffers by the operators around the routed layer, on the CPU: every bad call ends before any GPU
work, and the good ones have no rows."""
import pytest

import quantized_expert_gemv_amd as q

F = 1 << 40          # a fake aligned pointer: never dereferenced, every call below is refused
SHAPE = -2
F16, F32 = 1, 2
ROWS, COLS = 4, 256
ROW = 2 * COLS       # bytes of an fp16 row


def norm(**change):
    """gale_add_rms_norm on buffers 1 MiB apart, fp16, with all outputs; `change` moves some of them."""
    a = {"x": F, "x_stride": COLS, "res": F + (1 << 20), "res_stride": COLS, "dtype": F16, "rows": ROWS, "cols": COLS,
         "w": F + (2 << 20), "w_dtype": F16, "eps": 1e-6, "sum": F + (3 << 20), "y": F + (4 << 20), "y_dtype": F16, "fmt": 2,
         "codes": F + (5 << 20), "scales": F + (6 << 20)}
    a.update(change)
    st = q.lib().gale_add_rms_norm(*a.values(), None)
    return st, q.lib().gale_last_error().decode()


@pytest.mark.parametrize("change", [
    {"y": F, "x_stride": COLS + 1},                             # in place needs rows stored back to back
    {"y": F + (1 << 20), "res_stride": 300},
    {"y": F, "y_dtype": F32},                                   # and the input's type
    {"y": F + ROW},                                             # one row behind x
    {"y": F - ROW * ROWS + 2},                                  # its last element is x's first
    {"y": F + ROW * ROWS - 2},
    {"sum": F + 2},
    {"sum": F + (1 << 20) + ROW},
    {"sum": F + (2 << 20)},                                     # the weight
    {"y": F + (2 << 20) + ROW - 2},
    {"y": F + (3 << 20)},                                       # sum and y
    {"codes": F}, {"codes": F + (4 << 20)}, {"scales": F + (3 << 20) + 4}, {"scales": F + (5 << 20)},
    {"codes": F + (2 << 20)},
    {"sum": F, "y": F},
    {"x_stride": 10 * COLS, "y": F + 30 * ROW},                 # y begins at x's last row
])
def test_norm_refuses_overlaps(change):
    st, error = norm(**change)
    assert st == SHAPE and "overlap" in error or "in place" in error, change


def test_norm_overlaps_of_no_rows_are_none():
    assert norm(rows=0, y=F, sum=F)[0] == 0
