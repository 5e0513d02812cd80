"""The bars of w4_model on models of the kernels' roundings: the kernels' own pass, an H of bf16's
eight bits or blocks of twelve bits do not -- no GPU."""
import numpy as np
import pytest

import w4_model as model
import w4_ref


@pytest.mark.parametrize("act", ["relu", "swiglu"])
@pytest.mark.parametrize("d,dff", [(512, 896), (256, 2064)])
def test_what_the_bars_let_through(d, dff, act):
    w = model.matrices(model.experts(1, d, dff, 64, act, seed=d), 0, 64)
    x = model.rows(40, d, seed=1)
    want = model.ffn(x, *w, act)

    def worst(lost, x_round, h_round):
        err = model.rms(model.ffn(x, *w, act, x_round, h_round) - want)
        return (err / model.allowed(want, lost)).max(), (err / model.allowed(want, lost)).min()

    ints = [lambda v, b=b: model.to_blocks(v, b) for b in (64, 128)]
    assert worst(model.MANY, None, lambda h: model.to_bits(h, 11))[0] < 1
    assert worst(model.MANY, None, lambda h: model.to_bits(h, 8))[1] > 1     # in every row
    assert worst(model.FEW, ints[0], ints[0])[0] < 1 and worst(model.FEW, ints[1], ints[1])[0] < 1
    assert worst(model.FEW, ints[0], lambda h: model.to_bits(h, 8))[1] > 1
    coarse = lambda v: model.to_blocks(v, 64, levels=127)   # noqa: E731  (bytes)
    assert worst(model.FEW, coarse, ints[0])[1] > 1 and worst(model.FEW, ints[0], coarse)[1] > 1


@pytest.mark.parametrize("size,lost", [(300, 2.7e-3), (1000, 8.9e-3)])
def test_what_an_outlier_costs_a_block(size, lost):
    # one value of a block `size` times the others', which meets zero weights: the others keep the bits
    # that its unit leaves them, size / 32512 / sqrt 12 of their RMS
    assert abs(size / 32512 / np.sqrt(12) - lost) < 0.02 * lost
    W = model.experts(1, 512, 896, 64, "relu", seed=2)
    W["w1"][0][:, :, 5::64] = 0
    w = model.matrices(W, 0, 64)
    x = model.rows(40, 512, seed=3)
    x[:, 5::64] = size
    want = model.ffn(x, *w, "relu")
    err = model.ffn(x, *w, "relu", lambda v: model.to_blocks(v, 64), lambda h: model.to_blocks(h, 64)) - want
    # over all rows (a row's few hundred errors of x are common to its outputs): the rounding of y taken off in squares
    beside = np.sqrt(((err ** 2).mean() - ((w4_ref.bf16(want) - want) ** 2).mean()) / (want ** 2).mean())
    assert abs(beside - lost) < 0.2 * lost
