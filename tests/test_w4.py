"""The fp64 definition of 4-bit weights (w4_ref) on worked values, and the argument
checks of the 4-bit entry points -- no GPU: every refused call fails on the host."""
import ctypes

import numpy as np
import pytest

import w4_ref
from mixture_experts_sparse_b200 import native as nat

P = ctypes.c_void_p
OK, MIS = P(0x1000), P(0x1008)


def test_worked_group():
    # max 3.5 -> scale 0.5; ties go to the even code
    w = np.zeros((1, 32))
    w[0, :7] = [3.5, -3.5, 0.25, 0.75, -0.25, 1.2, -1.3]
    q, s = w4_ref.quantize(w, 32)
    assert s[0, 0] == 0.5 and list(q[0, :8]) == [7, -7, 0, 2, 0, 2, -3, 0]
    z, s0 = w4_ref.quantize(np.zeros((2, 48)), 32)
    assert not z.any() and s0.shape == (2, 2) and not s0.any()


def test_layout():
    q = np.full((1, 144), 0, np.int8)
    q[0, 0], q[0, 1], q[0, 8], q[0, 32], q[0, 128] = 1, 2, 3, 4, 5
    words = w4_ref.pack(q).view(np.uint32)[0]
    assert words.size == 32 and w4_ref.pack(q).shape[1] == nat.moe_w4_row_bytes(144) == 128
    assert words[0] == 0x888A8889 and words[4] == 0x8888888B and words[1] == 0x8888888C and words[16] == 0x8888888D
    assert words[31] == 0x88888888   # past K: zero weights
    assert [nat.moe_w4_row_bytes(k) for k in (16, 128, 1040, 4096)] == [64, 64, 576, 2048]


def test_rounding_to_bf16_is_not_doubled():
    # just above a bf16 tie: an fp32 rounding in between would land on the tie
    tie = 1 + 2.0 ** -8
    assert w4_ref.bf16(tie) == 1.0 and w4_ref.bf16(tie + 2.0 ** -30) == 1 + 2.0 ** -7


@pytest.mark.parametrize("a,status", [
    ((-1, 4, 64, 32, "f32"), nat.MOE_ERR_INVALID_ARG), ((1, -4, 64, 32, "f32"), nat.MOE_ERR_INVALID_ARG),
    ((1, 4, 0, 32, "f32"), nat.MOE_ERR_INVALID_ARG), ((1, 4, 72, 32, "f32"), nat.MOE_ERR_UNSUPPORTED),
    ((1, 4, 64, 16, "f32"), nat.MOE_ERR_UNSUPPORTED), ((1, 4, 64, 96, "bf16"), nat.MOE_ERR_UNSUPPORTED),
    ((1 << 31, 1, 64, 32, "f32"), nat.MOE_ERR_UNSUPPORTED), ((1 << 20, 1 << 20, 64, 32, "f32"), nat.MOE_ERR_UNSUPPORTED),
    ((1, 4, 1 << 25, 32, "f32"), nat.MOE_ERR_UNSUPPORTED)])
def test_bad_matrices_are_refused(a, status):
    m, r, k, g, dt = a
    for fn in (nat.lib().moe_quantize_w4, nat.lib().moe_dequantize_w4):
        assert fn(m, r, k, g, nat._dt(dt), OK, OK, OK, None) == status


def test_bad_matrix_pointers_are_refused():
    for fn in (nat.lib().moe_quantize_w4, nat.lib().moe_dequantize_w4):
        for i in range(3):
            for bad in (None, MIS):
                p = [OK, OK, OK]
                p[i] = bad
                assert fn(1, 4, 64, 32, 0, *p, None) == nat.MOE_ERR_INVALID_ARG
        assert fn(1, 4, 64, 32, 7, OK, OK, OK, None) == nat.MOE_ERR_INVALID_ARG
        assert fn(0, 4, 64, 32, 0, None, None, None, None) == nat.MOE_OK   # nothing to do
    assert nat.moe_w4_row_bytes(-1) == 0


NAMES = ("xe", "offsets", "q1", "s1", "b1", "q3", "s3", "b3", "q2", "s2", "b2", "ye")


def _ffn(cfg, group=64, ws=OK, nbytes=None, **over):
    p = dict.fromkeys(NAMES, OK)
    p.update(over)
    nbytes = nat.moe_w4_workspace_bytes(cfg) if nbytes is None else nbytes
    return nat.lib().moe_expert_ffn_w4(ctypes.byref(cfg), group, *[p[n] for n in NAMES], ws, nbytes, None)


def test_bad_expert_calls_are_refused():
    cfg = nat.config(4, 128, 256, 8, 2, 4, "bf16", "swiglu")
    for name in ("xe", "offsets", "q1", "s1", "q3", "s3", "q2", "s2", "ye"):
        assert _ffn(cfg, **{name: None}) == nat.MOE_ERR_INVALID_ARG, name
    for name in NAMES:
        assert _ffn(cfg, **{name: MIS}) == nat.MOE_ERR_INVALID_ARG, name
    assert _ffn(cfg, group=48) == nat.MOE_ERR_UNSUPPORTED
    assert _ffn(nat.config(4, 128, 256, 8, 2, 4, "f32", "swiglu"), nbytes=1 << 40) == nat.MOE_ERR_UNSUPPORTED
    assert _ffn(nat.config(4, 120, 256, 8, 2, 4)) == nat.MOE_ERR_UNSUPPORTED
    # too many weights for 32-bit counts of pipeline stages; rows longer than a launch covers
    assert _ffn(nat.config(4, 1 << 21, 1 << 18, 8, 1, 4), nbytes=1 << 60) == nat.MOE_ERR_UNSUPPORTED
    assert _ffn(nat.config(4, (1 << 23) + 16, 256, 8, 1, 4), nbytes=1 << 60) == nat.MOE_ERR_UNSUPPORTED
    assert _ffn(nat.config(-4, 128, 256, 8, 2, 4)) == nat.MOE_ERR_INVALID_ARG
    need = nat.moe_w4_workspace_bytes(cfg)
    assert need > nat.moe_workspace_bytes(cfg) and nat.moe_w4_workspace_bytes(nat.config(4, 128, 256, 8, 2, 4, "f32")) == 0
    assert _ffn(cfg, nbytes=need - 1) == _ffn(cfg, ws=None) == _ffn(cfg, ws=MIS) == nat.MOE_ERR_WORKSPACE
    # ReLU experts have no third matrix; no capacity: nothing is launched
    relu0 = nat.config(4, 128, 256, 8, 2, 0)
    assert _ffn(relu0, q3=None, s3=None, b1=None, b3=None, b2=None, xe=None, ye=None) == nat.MOE_OK


def test_bad_forward_calls_are_refused():
    cfg = nat.config(4, 128, 256, 8, 2, 4, "bf16", "swiglu")

    def fwd(group=64, nbytes=None, **over):
        n = ("x", "w_r", "b_r", "q1", "s1", "b1", "q3", "s3", "b3", "q2", "s2", "b2", "out")
        p = dict.fromkeys(n, OK)
        p.update(over)
        nbytes = nat.moe_w4_workspace_bytes(cfg) if nbytes is None else nbytes
        return nat.lib().moe_forward_w4(ctypes.byref(cfg), group, *[p[q] for q in n], *[None] * 10, OK, nbytes, None)

    for name in ("x", "w_r", "q1", "s1", "q3", "s3", "q2", "s2", "out"):
        assert fwd(**{name: None}) == nat.MOE_ERR_INVALID_ARG, name
    assert fwd(group=0) == nat.MOE_ERR_UNSUPPORTED
    assert fwd(nbytes=nat.moe_workspace_bytes(cfg)) == nat.MOE_ERR_WORKSPACE   # the bf16 layer's is too small


def test_names_of_types():
    torch = pytest.importorskip("torch")
    for name in ("f32", nat.MOE_F32, torch.float32):
        assert nat._dt(name) == nat.config(4, 16, 16, 2, 1, 4, name).dtype == nat.balance_config(4, 2, 1, 1, name).dtype == nat.MOE_F32
    for name in ("bf16", nat.MOE_BF16, torch.bfloat16):
        assert nat._dt(name) == nat.config(4, 16, 16, 2, 1, 4, name).dtype == nat.balance_config(4, 2, 1, 1, name).dtype == nat.MOE_BF16
    # taken for fp32, each of these would have the kernels read and write past a buffer's end
    for name in ("bfloat16", "f16", "fp16", torch.float16, torch.int32, np.float32, 2, -1, None):
        for call in (lambda: nat.config(4, 16, 16, 2, 1, 4, name), lambda: nat.balance_config(4, 2, 1, 1, name),
                     lambda: nat.moe_quantize_w4(1, 4, 64, 32, name, None, None, None, 0),
                     lambda: nat.moe_dequantize_w4(1, 4, 64, 32, name, None, None, None, 0)):
            with pytest.raises(ValueError):
                call()
