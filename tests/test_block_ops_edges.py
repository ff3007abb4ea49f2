"""Refusals of overlapping buffers by the operators around the routed layer, on the CPU: every bad call ends before any GPU
work, and the good ones have no rows."""
import random

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


M, N, K = 5, 64, 256


def gemm(**change):
    """gale_mx_gemm of fp16 results on buffers 1 MiB apart, y and add in rows of 200."""
    a = {"m": M, "n": N, "k": K, "a": F, "as": F + (1 << 20), "a_fmt": 2, "w": F + (2 << 20), "ws": F + (3 << 20),
         "add": F + (4 << 20), "add_stride": 200, "y": F + (5 << 20), "y_dtype": F16, "y_stride": 200}
    a.update(change)
    st = q.lib().gale_mx_gemm(*a.values(), None)
    return st, q.lib().gale_last_error().decode()


Y = F + (4 << 20)        # add's place


@pytest.mark.parametrize("change", [
    {"y": Y + 2}, {"y": Y - 2}, {"y": Y + 2 * (N - 1)}, {"y": Y - 2 * (N - 1)},          # the same stride, columns in common
    {"y": Y + 2 * 400 + 2 * 63}, {"y": Y + 2 * 200 - 2}, {"y": Y + 2 * 800}, {"y": Y - 2 * 800 + 126},
    {"y": Y, "y_stride": 201}, {"y": Y + 2 * 64, "y_stride": 250}, {"y": Y + 2 * 130, "y_stride": 64},   # other strides
    {"y": Y - 2 * 64, "y_stride": 264}, {"add": None, "y": F}, {"y": F + M * 256 - 2}, {"y": F + (1 << 20) + 16},
    {"y": F + (2 << 20) + N * 128 - 2}, {"y": F + (3 << 20) - 2 * 200 - 2}, {"m": 1, "y": Y + 126}, {"m": 1, "y": Y - 126},
])
def test_gemm_refuses_overlaps(change):
    st, error = gemm(**change)
    assert st == SHAPE and ("overlaps" in error or "in place" in error), change


def test_overlaps_are_found_as_element_by_element():
    """Random rows of add and y, of one stride or two, against the sets of their elements: where these meet, the call is
    refused."""
    rng, met = random.Random(5), 0
    for _ in range(4000):
        n, sx, sy = rng.randint(1, 6), rng.randint(6, 20), rng.randint(6, 20)
        sy = sx if rng.random() < 0.5 else sy
        rows, at = rng.randint(1, 5), rng.randint(-60, 60)
        x = {r * sx + c for r in range(rows) for c in range(n)}
        y = {at + r * sy + c for r in range(rows) for c in range(n)}
        if at == 0 or not x & y:
            continue
        met += 1
        st, error = gemm(m=rows, n=n, y=Y + 2 * at, add_stride=sx, y_stride=sy)
        assert st == SHAPE and "overlaps" in error, (rows, n, sx, sy, at)
    assert met > 500


def test_norm_refuses_an_infinite_eps():
    st, error = norm(eps=float("inf"))
    assert st == SHAPE and "eps" in error


@pytest.mark.parametrize("name,two", [("gale_mx_quantize", 1), ("gale_mx_swiglu_quantize", 2)])
@pytest.mark.parametrize("codes,scales", [(F, F + (2 << 20)), (F + 16, F + (2 << 20)), (F - 3 * 64 - 16, F + (2 << 20)),
                                          (F + (2 << 20), F + 8), (F + (2 << 20), F + (2 << 20) + 4), (F + (2 << 20), F - 12)])
def test_quantisers_refuse_overlaps(name, two, codes, scales):
    st = getattr(q.lib(), name)(F, F16, 300 * two, 4, 128, 1, codes, scales, None)
    assert st == SHAPE and "overlaps" in q.lib().gale_last_error().decode()


@pytest.mark.parametrize("y", [F, F + 3 * 64, F - 3 * 600 - 254, F + (1 << 20), F + (1 << 20) + 12])
def test_dequantiser_refuses_overlaps(y):
    st = q.lib().gale_mx_dequantize(F, F + (1 << 20), 1, 4, 128, y, F16, 300, None)
    assert st == SHAPE and "overlaps" in q.lib().gale_last_error().decode()


@pytest.mark.parametrize("bias,idx,w", [
    (None, F, F + (2 << 20)), (None, F + (1 << 20), F + 3 * 1200 + 1020), (None, F + (1 << 20), F + (1 << 20) + 124),
    (F + (3 << 20), F + (3 << 20) + 1020, F + (1 << 20)), (F + (3 << 20), F + (1 << 20), F + (3 << 20) - 124)])
def test_router_refuses_overlaps(bias, idx, w):
    st = q.lib().gale_route_scored(F, F32, 300, 4, 256, bias, 2, 8, 4, 2, 8, 1, 1.0, idx, w, None)
    assert st == SHAPE and "overlaps" in q.lib().gale_last_error().decode()
