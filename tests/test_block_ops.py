"""The operators around the routed layer on the CPU: pins of their oracle, sizes, and every refusal of a bad call
before any GPU work."""
import numpy as np
import pytest
import torch

import quantized_expert_gemv_amd as q
from oracle import block_oracle as O

F = 1 << 40          # a fake aligned pointer: never dereferenced, every call below is refused
NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED = -1, -2, -3, -4, -5, -6


# ---- the oracle --------------------------------------------------------------------------------------------------
def test_element_tables_are_the_formats():
    f8 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.E4M3, f8) and O.E4M3[-1] == 448
    assert list(O.E2M1) == sorted({(1 + m / 2) * 2.0 ** (e - 1) for e in (1, 2, 3) for m in (0, 1)} | {0, 0.5})


@pytest.mark.parametrize("fmt", [1, 2])
def test_rounding_is_to_nearest_even(fmt):
    table = O.TABLE[fmt]
    for i in range(len(table) - 1):
        mid = (table[i] + table[i + 1]) / 2
        d = (table[i + 1] - table[i]) / 64
        got = O.mx_round(np.array([table[i], mid - d, mid, mid + d]), table)
        assert list(got) == [i, i, i + i % 2, i + 1]


@pytest.mark.parametrize("fmt,top", [(1, 6.0), (2, 448.0)])
def test_scale_is_the_smallest_that_does_not_saturate(fmt, top):
    x = np.zeros((1, 128))
    x[0, 0], x[0, 32], x[0, 64], x[0, 96] = top, np.nextafter(top, 1e9), top / 2, 1e-60
    codes, scales = O.mx_quantize(x, fmt)
    assert list(scales[0]) == [127, 128, 126, 0]
    v = O.mx_values(codes, scales, fmt, 128)
    assert v[0, 0] == top and v[0, 32] in (top, 2 * O.TABLE[fmt][np.searchsorted(O.TABLE[fmt], top / 2)]) and v[0, 64] == top / 2
    assert v[0, 96] == 0.0


def test_route_oracle_against_closed_forms():
    l = np.array([[1.0, 3.0, 2.0, 3.0]])
    idx, w = O.route_scored(l, 2)
    assert list(idx[0]) == [1, 3] and np.allclose(w, 0.5)
    idx, w = O.route_scored(l, 2, renormalize=False, scale=2.0)
    assert np.allclose(w, 2 * np.exp(3) / np.exp(l).sum())
    # the bias moves the choice, the weights stay the scores
    idx, w = O.route_scored(l, 1, score="sigmoid", bias=[5, 0, 0, 0], renormalize=False)
    assert idx[0, 0] == 0 and np.isclose(w[0, 0], 1 / (1 + np.exp(-1)))
    # two groups: the sum of two beats the single best only under top2
    l = np.array([[2.0, -9.0, 1.5, 1.4]])
    assert O.route_scored(l, 1, score="sigmoid", n_groups=2, keep_groups=1, group_score="top2")[0][0, 0] == 2
    assert O.route_scored(l, 1, score="sigmoid", n_groups=2, keep_groups=1, group_score="max")[0][0, 0] == 0
    # nothing to choose
    idx, w = O.route_scored(np.full((1, 4), -np.inf), 2)
    assert list(idx[0]) == [-1, -1] and not w.any()


# ---- sizes and refusals ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("cols,groups", [(1, 1), (32, 1), (128, 1), (129, 2), (4096, 32), (65536, 512)])
def test_row_sizes(cols, groups):
    L = q.lib()
    assert L.gale_mx_code_bytes(q.GALE_MX_E2M1, cols) == 64 * groups
    assert L.gale_mx_code_bytes(q.GALE_MX_E4M3, cols) == 128 * groups
    assert L.gale_mx_scale_bytes(cols) == 4 * groups
    mx = q.MXTensor.empty(3, cols, q.GALE_MX_E2M1, "cpu")
    assert mx.rows == 3 and mx.codes.shape[1] == 64 * groups


def test_row_sizes_of_bad_arguments_are_zero():
    L = q.lib()
    for cols in (0, -1, 65537):
        assert L.gale_mx_code_bytes(q.GALE_MX_E2M1, cols) == 0 and L.gale_mx_scale_bytes(cols) == 0
    assert L.gale_mx_code_bytes(3, 128) == 0


def _refused(name, good, changes):
    f = getattr(q.lib(), name)
    for want, change in changes:
        args = list(good)
        for i, v in change.items():
            args[i] = v
        assert f(*args) == want, (name, change)
        assert name in q.lib().gale_last_error().decode()


def test_route_scored_refusals():
    # logits, dtype, stride, n_tok, E, bias, score, groups, keep, rule, k, renorm, scale, idx, w, stream
    good = [F, 2, 256, 4, 256, None, 2, 8, 4, 2, 8, 1, 1.0, F, F, None]
    _refused("gale_route_scored", good, [
        (DTYPE, {1: 4}), (SHAPE, {2: 255}), (SHAPE, {3: -1}), (SHAPE, {4: 0}), (SHAPE, {4: 513, 2: 600}),
        (UNSUPPORTED, {6: 0}), (UNSUPPORTED, {6: 3}), (SHAPE, {7: 0}), (SHAPE, {7: 7}), (SHAPE, {7: 128}), (SHAPE, {8: 0}),
        (SHAPE, {8: 9}), (UNSUPPORTED, {9: 0}), (SHAPE, {10: 0}), (SHAPE, {10: 9}), (SHAPE, {7: 64, 8: 1, 10: 5}),
        (NULL, {0: None}), (NULL, {13: None}), (NULL, {14: None}), (ALIGN, {0: F + 2}), (ALIGN, {5: F + 2}),
        (ALIGN, {13: F + 1}), (ALIGN, {14: F + 2})])
    good[3] = 0
    assert q.lib().gale_route_scored(*good) == 0          # no tokens: nothing to do


@pytest.mark.parametrize("name,two", [("gale_mx_quantize", 1), ("gale_mx_swiglu_quantize", 2)])
def test_quantize_refusals(name, two):
    # x, dtype, stride, rows, cols, fmt, codes, scales, stream
    good = [F, 1, 256 * two, 4, 256, 1, F, F, None]
    _refused(name, good, [
        (DTYPE, {1: 0}), (DTYPE, {5: 0}), (DTYPE, {5: 3}), (SHAPE, {2: 256 * two - 1}), (SHAPE, {3: -1}), (SHAPE, {3: 1 << 31}),
        (SHAPE, {4: 0}), (SHAPE, {4: 65537, 2: 1 << 20}), (NULL, {0: None}), (NULL, {6: None}), (NULL, {7: None}),
        (ALIGN, {0: F + 1}), (ALIGN, {6: F + 8}), (ALIGN, {7: F + 2})])
    good[3] = 0
    assert getattr(q.lib(), name)(*good) == 0


def test_dequantize_refusals():
    # codes, scales, fmt, rows, cols, y, dtype, stride, stream
    good = [F, F, 1, 4, 256, F, 1, 256, None]
    _refused("gale_mx_dequantize", good, [
        (DTYPE, {2: 0}), (DTYPE, {6: 0}), (SHAPE, {7: 255}), (SHAPE, {3: -1}), (SHAPE, {4: 0}), (NULL, {0: None}),
        (NULL, {1: None}), (NULL, {5: None}), (ALIGN, {0: F + 4}), (ALIGN, {1: F + 1}), (ALIGN, {5: F + 1})])


def test_gemm_refusals():
    # m, n, k, a, as, a_fmt, w, ws, add, add_stride, y, y_dtype, y_stride, stream
    good = [4, 64, 256, F, F, 2, F, F, F, 64, F + 4096, 1, 64, None]
    _refused("gale_mx_gemm", good, [
        (SHAPE, {0: -1}), (SHAPE, {0: (1 << 20) + 1}), (SHAPE, {1: 0}), (SHAPE, {1: (1 << 20) + 1, 9: 1 << 21, 12: 1 << 21}),
        (SHAPE, {2: 0}), (SHAPE, {2: 65537}), (DTYPE, {5: 0}), (DTYPE, {11: 7}), (SHAPE, {12: 63}), (SHAPE, {9: 63}),
        (SHAPE, {8: F + 4096, 9: 65}), (NULL, {3: None}), (NULL, {4: None}), (NULL, {6: None}), (NULL, {7: None}),
        (NULL, {10: None}), (ALIGN, {3: F + 8}), (ALIGN, {4: F + 2}), (ALIGN, {6: F + 1}), (ALIGN, {7: F + 1}),
        (ALIGN, {8: F + 1}), (ALIGN, {10: F + 1})])
    good[0] = 0
    assert q.lib().gale_mx_gemm(*good) == 0


def test_norm_refusals():
    # x, x_stride, res, res_stride, dtype, rows, cols, w, w_dtype, eps, sum, y, y_dtype, fmt, codes, scales, stream
    G = F + (1 << 20)
    good = [F, 256, G, 256, 1, 4, 256, F, 1, 1e-6, F + 4096, F + 8192, 1, 2, F, F, None]
    _refused("gale_add_rms_norm", good, [
        (DTYPE, {4: 0}), (DTYPE, {8: 0}), (DTYPE, {12: 0}), (DTYPE, {13: 0}), (SHAPE, {1: 255}), (SHAPE, {3: 255}),
        (SHAPE, {5: -1}), (SHAPE, {6: 0}), (SHAPE, {6: 16385, 1: 1 << 20, 3: 1 << 20}), (SHAPE, {9: -1.0}),
        (SHAPE, {9: float("nan")}), (NULL, {14: None}), (NULL, {15: None}), (NULL, {0: None}),
        (NULL, {11: None, 14: None, 15: None}), (SHAPE, {10: F, 1: 257}), (SHAPE, {10: G, 3: 300}), (ALIGN, {0: F + 1}),
        (ALIGN, {2: F + 1}), (ALIGN, {7: F + 1}), (ALIGN, {10: F + 1}), (ALIGN, {11: F + 1}), (ALIGN, {14: F + 8}),
        (ALIGN, {15: F + 2})])
    good[5] = 0
    assert q.lib().gale_add_rms_norm(*good) == 0


def test_given_layer_refusals():
    # hidden, inter, experts, E, idx, w, k, x, n_tok, y, ws, ws_bytes, flags, stream
    good = [4096, 2048, F, 256, F, F, 6, F, 1, F, F, 1 << 30, 0, None]
    _refused("gale_moe_layer_fwd_given", good, [
        (SHAPE, {0: 4000}), (SHAPE, {3: 513}), (SHAPE, {6: 9}), (SHAPE, {8: 0}), (NULL, {4: None}), (NULL, {5: None}),
        (NULL, {2: None}), (NULL, {7: None}), (NULL, {9: None}), (NULL, {10: None}), (ALIGN, {4: F + 2}),
        (ALIGN, {5: F + 2}), (WORKSPACE, {11: 16})])


def test_bf16_stays_refused_elsewhere():
    assert q.lib().gale_fwht1024(F, F, 1, 1024, q.GALE_BF16, q.GALE_BF16, None) == DTYPE


def test_binding_refusals():
    x = torch.zeros(4, 256, dtype=torch.float16)
    with pytest.raises(ValueError):
        q.mx_quantize(x)                                        # not on a GPU
    with pytest.raises(ValueError):
        q.MXTensor(torch.zeros(4, 100, dtype=torch.uint8), torch.zeros(4, 8, dtype=torch.uint8), 256, q.GALE_MX_E2M1)
    with pytest.raises(ValueError):
        q.MXTensor(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 8, dtype=torch.uint8), 256, 5)
    a, w = q.MXTensor.empty(4, 256, q.GALE_MX_E4M3, "cpu"), q.MXTensor.empty(8, 256, q.GALE_MX_E4M3, "cpu")
    with pytest.raises(ValueError):
        q.mx_gemm(a, w)                                         # w must be 4 bits
    w = q.MXTensor.empty(8, 384, q.GALE_MX_E2M1, "cpu")
    with pytest.raises(ValueError):
        q.mx_gemm(a, w)                                         # other columns
    w = q.MXTensor.empty(8, 256, q.GALE_MX_E2M1, "cpu")
    for bad in (torch.zeros(4, 7), torch.zeros(8, 4).T, torch.zeros(1, 8).expand(4, 8)):
        with pytest.raises(ValueError):
            q.mx_gemm(a, w, out=bad)
    with pytest.raises(ValueError):
        q.mx_gemm(a, w, add=torch.zeros(4, 8), out=torch.zeros(4, 8, dtype=torch.float16))
    with pytest.raises(ValueError):
        q.mx_swiglu_quantize(x[:, :255])
    with pytest.raises(ValueError):
        q.add_rms_norm(x, None, residual=x.float())
    with pytest.raises(ValueError):
        q.add_rms_norm(x, torch.ones(255))
    with pytest.raises(ValueError):
        q.add_rms_norm(x, None, sum_out=torch.zeros(4, 256))
    with pytest.raises(ValueError):
        q.route_scored(x, 4, score="relu")
    with pytest.raises(ValueError):
        q.route_scored(x, 4, bias=torch.zeros(256, dtype=torch.float16))
    with pytest.raises(ValueError):
        q.route_scored(x, 4, out=(torch.zeros(4, 4), torch.zeros(4, 4)))
    with pytest.raises(ValueError):
        q.route_scored(x.double(), 4)
