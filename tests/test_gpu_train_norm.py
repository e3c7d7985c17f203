"""GPU tests of layer norm's sums over many rows, and of long rows in number.

Tolerance of the column sums.  A block adds up its rows one by one, at least one block per SM (or
32 slices of the rows past 8192 elements); then 32 slices of at most 8 * SMs / 32 blocks are added one by
one, then the slices: each addition is off by u32 of the magnitudes so far, and a term by 4 u32.  That is
far less than any one row adds, so a row left out or added twice shows."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_19_gb300.workload import to_f64
from oracle import train_ref
from tests.test_gpu_train import check_ln, ln_inputs, within

pytestmark = pytest.mark.gpu
U16, U32 = 2.0 ** -8, 2.0 ** -24
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def train():
    from mixture_experts_layer_19_gb300 import train
    yield train
    assert train.device_status(0) == 0


@pytest.mark.parametrize("rows,d,xt", [(10007, 64, BF), (10007, 64, F32), (3001, 257, BF), (5000, 1001, F32),
                                       (2500, 691, F32), (2049, 1024, BF), (4096, 2048, BF), (1000, 7168, F32), (700, 9001, BF),
                                       (700, 9001, F32), (2000, 8200, BF), (2000, 8200, F32), (33, 8200, BF)])
def test_column_sums(train, rows, d, xt):
    x, w, _, dy = ln_inputs(rows, d, xt, F32, seed=rows + d)
    X, DY = to_f64(x), to_f64(dy)
    _, mean, rstd = train.layer_norm_forward(x.to(DEV), w.to(DEV))
    _, dw, db = train.layer_norm_backward(dy.to(DEV), x.to(DEV), w.to(DEV), mean, rstd)
    sm, sr = to_f64(mean), to_f64(rstd)
    _, rw, rb = train_ref.layer_norm_backward(DY, X, to_f64(w), sm, sr)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    blocks = min(rows, sms if d <= 8192 else 32)
    chain = (-(-rows // blocks) + -(-8 * sms // 32) + 32) * U32
    n = np.abs(X - sm[:, None]) * sr[:, None]
    off = (chain + 4 * U32) * (np.abs(DY) * n).sum(0), chain * np.abs(DY).sum(0)
    # a row's own share of db is over the bound in all but a few columns
    assert (np.median(np.abs(DY), axis=0) > 2 * off[1]).mean() > 0.9
    within(dw, rw, off[0] + U32 * np.abs(rw))
    within(db, rb, off[1] + U32 * np.abs(rb))


@pytest.mark.parametrize("rows,d,xt", [(700, 9001, BF), (700, 9001, F32), (2000, 8200, BF), (2000, 8200, F32),
                                       (2000, 12288, BF), (700, 16384, BF), (700, 12288, F32)])
def test_long_rows_in_number(train, rows, d, xt):
    """More rows than blocks, where rows are read again, and bf16 rows of up to 16384 that four warps hold."""
    check_ln(train, *ln_inputs(rows, d, xt, F32, seed=rows))


@pytest.mark.parametrize("rows,d", [(3, 64), (3, 691), (3, 1001), (3, 7168), (3, 8200), (3, 9001), (2000, 64),
                                    (2000, 256), (2000, 691), (2000, 2051), (2000, 7168), (700, 9001)])
@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("value", [3.3, 1000.0, 12345.6, 1e6])
def test_rows_of_one_value(train, rows, d, xt, value):
    """The mean of such a row is its value, and nothing is left of it.  The first mean is off by at most 512 u32
    of the value (its sum's chain); the mean of the deviations, all the same, restores it to the bit, since
    that is off by 512 u32 of 512 units of the last place, less than half of one."""
    x = torch.full((rows, d), value, device=DEV).to(xt)
    w, b = torch.full((d,), 1.5, device=DEV), torch.full((d,), 0.25, device=DEV)
    y, mean, rstd = train.layer_norm_forward(x, w, b)
    assert (mean == x[0, 0].float()).all() and (y == 0.25).all()
    # the deviations' squares cancel to 512 u32 of (512 u32 value)^2
    off = 512 * U32 * (512 * U32 * value) ** 2 + 4 * U32 * 1e-5
    assert ((rstd.double() ** -2 - 1e-5).abs() <= off + 4 * U32 * 1e-5).all()


@pytest.mark.parametrize("rows,d", [(7, 64), (7, 1001), (7, 7168), (7, 9001), (2000, 256), (2000, 1001), (2000, 7168)])
def test_mean_far_from_zero(train, rows, d):
    """The mean is right to its last place (u32 of it, and the deviations' own chain), so a row's values are off
    by that much of the spread, and no more, however long the row."""
    x, w, b, _ = ln_inputs(rows, d, F32, F32, seed=d, shift=5000.0)
    X = to_f64(x)
    ry, rm, rr = train_ref.layer_norm(X, to_f64(w), to_f64(b), 1e-5)
    y, mean, rstd = train.layer_norm_forward(x.to(DEV), w.to(DEV), b.to(DEV))
    e = 512 * U32
    spread = np.abs(X - rm[:, None])
    dm = 2 * U32 * np.abs(rm) + e * (spread.mean(1) + 512 * U32 * np.abs(rm))
    within(mean, rm, dm)
    n_off = (e * spread + dm[:, None]) * rr[:, None]
    y_off = n_off * np.abs(to_f64(w)) + 8 * U32 * (np.abs(ry) + np.abs(to_f64(b)))
    within(y, ry, y_off)
