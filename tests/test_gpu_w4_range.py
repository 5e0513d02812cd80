"""4-bit experts on values near the ends of fp32's and bf16's range, in both kernels
(few and many rows), against fp64 within the bound of w4_ref.  The sums are scaled by
powers of two inside, which must not leave fp32 where the results do not."""
import numpy as np
import pytest

import w4_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from test_gpu_w4 import expert_values, make_experts, make_rows, run_ffn  # noqa: E402

MANY, FEW = [70, 200], [3, 2]


def scaled(W, dev, **powers):
    """Every scale of the named matrices times 2^power."""
    for n, p in powers.items():
        W[n] = (W[n][0], W[n][1] * 2.0 ** p)
        assert (np.abs(W[n][1]) >= 2.0 ** -126).all() and (np.abs(W[n][1]) < 2.0 ** 127).all()
        dev[n] = (dev[n][0], torch.from_numpy(W[n][1]).to(torch.bfloat16).cuda())


def check(W, x, y, off, group, act):
    xv = x.double().numpy()
    for e in range(len(off) - 1):
        rows = slice(off[e], off[e + 1])
        bias = [None if W[n] is None else W[n][e] for n in ("b1", "b3", "b2")]
        with np.errstate(over="ignore"):   # e^-u of a far negative u: silu is 0
            want, bound = w4_ref.ffn(xv[rows], *expert_values(W, e, group), *bias, act, 2.0 ** -11)
        assert (np.abs(want) < 2.0 ** 120).all() and np.median(np.abs(want)) > 2.0 ** -110
        err = np.abs(y.double().numpy()[rows] - want)
        assert (err <= bound).all(), f"expert {e}: {np.max(err / bound):.3g} of the bound"
        # two roundings to bf16 and spare, relative RMS (row by row, whatever their sizes)
        rms = np.sqrt((err ** 2).mean(1) / (want ** 2).mean(1))
        assert (rms < 3.5e-3).all(), f"expert {e}: relative RMS {rms.max():.2e}"


def case(act, rows, x_pow, group=64, bias=False, **powers):
    N, d, dff = len(rows), 256, 320
    off = np.concatenate([[0], np.cumsum(rows)]).tolist()
    W, dev = make_experts(N, d, dff, group, act, bias, seed=group)
    scaled(W, dev, **powers)
    x = (make_rows(off[-1], d).double() * 2.0 ** x_pow).to(torch.bfloat16)
    assert torch.isfinite(x).all()
    check(W, x, run_ffn(dev, x, off, N, d, dff, group, act, off[-1]), off, group, act)


@pytest.mark.parametrize("rows", [MANY, FEW])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("act,x_pow,powers", [
    # rows of x whose largest value is near 2^125, bf16's own largest being 2^128
    ("relu", 123, dict(w2=-60)), ("swiglu", 123, dict(w1=-100, w3=-60, w2=-40)),
    # weights near 2^-107
    ("relu", 30, dict(w1=-100)), ("swiglu", 60, dict(w1=-100, w3=-20)), ("relu", 40, dict(w2=-100)),
    # H near 2^121, its bound well past fp32
    ("swiglu", 62, dict(w2=-60)), ("relu", 20, dict(w1=100, w2=-60)),
    # both ends at once
    ("relu", 120, dict(w1=-100, w2=-10)), ("relu", -80, dict(w1=100, w2=20)),
    # blocks of x whose units are subnormal in the few-row kernel
    ("relu", -98, dict(w1=90))])
def test_far_powers_of_two(rows, act, x_pow, powers, group):
    case(act, rows, x_pow, group, **powers)


@pytest.mark.parametrize("rows", [MANY, FEW])
def test_rows_and_features_at_both_ends_of_one_tile(rows):
    # x from 2^-60 to 2^120 from row to row, weight rows from 2^-100 to 2^60 within the same tile
    N, d, dff, group = 2, 256, 320, 64
    W, dev = make_experts(N, d, dff, group, "relu", False, seed=3)
    rng = np.random.default_rng(5)
    W["w1"] = (W["w1"][0], W["w1"][1] * 2.0 ** rng.integers(-15, 1, (N, 1, dff)))
    W["w2"] = (W["w2"][0], W["w2"][1] * 2.0 ** rng.integers(-100, 1, (N, 1, d)))
    scaled(W, dev, w1=-20, w2=0)
    off = np.concatenate([[0], np.cumsum(rows)]).tolist()
    x = (make_rows(off[-1], d).double() * torch.from_numpy(2.0 ** rng.integers(0, 121, (off[-1], 1)))).to(torch.bfloat16)
    y = run_ffn(dev, x, off, N, d, dff, group, "relu", off[-1])
    xv = x.double().numpy()
    for e in range(N):
        r = slice(off[e], off[e + 1])
        want, bound = w4_ref.ffn(xv[r], *expert_values(W, e, group), None, None, None, "relu", 2.0 ** -11)
        # y below 2^-120 may be subnormal
        assert (np.abs(y.double().numpy()[r] - want) <= bound + 2.0 ** -126).all()
