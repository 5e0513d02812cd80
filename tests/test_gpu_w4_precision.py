"""The precision of the 4-bit expert kernels: every row's RMS error within the bar of w4_model,
which an H of bf16's eight bits or activations of ten bits do not meet (test_w4_precision)."""
import numpy as np
import pytest

import w4_model as model
import w4_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from test_gpu_w4 import run_ffn  # noqa: E402


def device(W):
    dev = {n: (None, None) if W[n] is None else (torch.from_numpy(w4_ref.pack(W[n][0])).cuda(),
                                                 torch.from_numpy(W[n][1]).to(torch.bfloat16).cuda()) for n in W}
    return dict(dev, b1=None, b3=None, b2=None)


def run(W, x, off, N, d, dff, group, act):
    y = run_ffn(device(W), torch.from_numpy(x).to(torch.bfloat16), off, N, d, dff, group, act, off[-1])
    return y.double().numpy()


@pytest.mark.parametrize("act", ["relu", "swiglu"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("d,dff,rows", [(512, 896, [3, 2]), (256, 2064, [0, 9, 16]), (512, 896, [70, 30]), (256, 2064, [150, 300])])
def test_every_rows_rms(d, dff, rows, group, act):
    N, off = len(rows), np.concatenate([[0], np.cumsum(rows)]).tolist()
    W = model.experts(N, d, dff, group, act, seed=d + group)
    x = model.rows(off[-1], d, seed=group)
    y = run(W, x, off, N, d, dff, group, act)
    lost = model.FEW if off[-1] <= 16 * N else model.MANY
    for e in range(N):
        r = slice(off[e], off[e + 1])
        if off[e] < off[e + 1]:
            want = model.ffn(x[r], *model.matrices(W, e, group), act)
            worst = (model.rms(y[r] - want) / model.allowed(want, lost)).max()
            assert worst <= 1, f"expert {e}: {worst:.3f} of the bar"


@pytest.mark.parametrize("size,lost", [(300, 2.7e-3), (1000, 8.9e-3)])
def test_outliers_that_meet_zero_weights(size, lost):
    # few rows: what test_w4_precision derives; a configuration with room for more takes x exactly
    N, d, dff, group = 4, 512, 896, 64
    W = model.experts(N, d, dff, group, "relu", seed=2)
    W["w1"][0][:, :, 5::64] = 0
    for rows, bar in ((10, 1.2 * lost), (30, model.MANY)):
        off = [rows * i for i in range(N + 1)]
        x = model.rows(off[-1], d, seed=3)
        x[:, 5::64] = size
        y = run(W, x, off, N, d, dff, group, "relu")
        err, noise, power = 0.0, 0.0, 0.0
        for e in range(N):
            r = slice(off[e], off[e + 1])
            want = model.ffn(x[r], *model.matrices(W, e, group), "relu")
            err += ((y[r] - want) ** 2).mean()
            noise += ((w4_ref.bf16(want) - want) ** 2).mean()
            power += (want ** 2).mean()
        # one per cent of the rounding of y: its samples
        assert err <= 1.01 * noise + bar ** 2 * power, (rows, np.sqrt(err / power))
