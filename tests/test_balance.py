"""The balance loss's fp64 definition (balance_ref) against the pinned oracle,
against central differences, and the argument checks of its entry points -- no
GPU: every refused call fails on the host."""
import ctypes

import numpy as np
import pytest

import balance_ref
import oracle
from mixture_experts_sparse_b200 import native as nat


def _batch(T, N, k, S, seed):
    rng = np.random.default_rng(seed)
    h = rng.standard_normal((T, N)) * 2
    idx = np.argsort(-h, axis=1)[:, :k].astype(np.int32)
    seqs = np.concatenate([[0], np.sort(rng.integers(0, T + 1, S - 1)), [T]]).astype(np.int32)
    return h, idx, seqs, (rng.random(T) < 0.7).astype(np.uint8)


def test_one_sequence_is_the_layers_own_loss():
    h, idx, _, _ = _batch(300, 12, 1, 1, 0)
    p, _ = balance_ref.softmax(h)
    got, counts, P, tokens = balance_ref.loss(h, idx, None, None, 0.01, 1.0)
    f, P0, aux = oracle.aux_loss(idx, p.astype(np.float32), 0.01)
    np.testing.assert_allclose(counts[0] / 300, f, rtol=0, atol=1e-15)
    np.testing.assert_allclose(P[0], P0, rtol=1e-6)
    np.testing.assert_allclose(got[0], aux, rtol=1e-6)
    np.testing.assert_allclose(got[1], oracle.z_loss(h.astype(np.float32)), rtol=1e-6)
    assert list(tokens) == [300, 300, 1]


@pytest.mark.parametrize("T,N,k,S", [(23, 5, 2, 4), (9, 3, 3, 1), (40, 17, 4, 9)])
def test_gradient_matches_central_differences(T, N, k, S):
    h, idx, seqs, mask = _batch(T, N, k, S, T)
    g, (alpha, zc) = (0.7, -1.3), (0.3, 0.2)
    _, counts, _, _ = balance_ref.loss(h, idx, mask, seqs, alpha, zc)
    d, _, _ = balance_ref.gradient(h, k, mask, seqs, alpha, zc, counts, g)
    eps = 1e-5
    for t, j in [(t, j) for t in range(0, T, 3) for j in range(N)]:
        hi, lo = h.copy(), h.copy()
        hi[t, j] += eps
        lo[t, j] -= eps
        num = np.dot(g, balance_ref.loss(hi, idx, mask, seqs, alpha, zc)[0]
                     - balance_ref.loss(lo, idx, mask, seqs, alpha, zc)[0]) / (2 * eps)
        # differences: truncation eps^2 f''' / 6 (|f'''| < 4 here) and rounding 2^-52 / eps
        assert abs(num - d[t, j]) <= 4 * eps * eps + 4 * 2.0 ** -52 / eps, (t, j)


P = ctypes.c_void_p
OK, MIS = P(0x1000), P(0x1008)


def _loss(cfg, logits=OK, idx=OK, mask=None, seqs=OK, loss=OK, counts=OK, P_=None, tokens=OK, ws=OK, nbytes=1 << 40):
    return nat.lib().moe_balance_loss(ctypes.byref(cfg), logits, idx, mask, seqs, loss, counts, P_, tokens, ws, nbytes,
                                      None)


def _grad(cfg, logits=OK, mask=None, seqs=OK, counts=OK, tokens=OK, dloss=None, dlogits=OK, accumulate=0):
    return nat.lib().moe_balance_loss_backward(ctypes.byref(cfg), logits, mask, seqs, counts, tokens, dloss, dlogits,
                                               accumulate, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), nat.MOE_ERR_INVALID_ARG), (dict(n_experts=0), nat.MOE_ERR_INVALID_ARG),
    (dict(top_k=0), nat.MOE_ERR_INVALID_ARG), (dict(top_k=9, n_experts=8), nat.MOE_ERR_INVALID_ARG),
    (dict(n_seqs=0), nat.MOE_ERR_INVALID_ARG), (dict(alpha=float("nan")), nat.MOE_ERR_INVALID_ARG),
    (dict(z_coef=float("inf")), nat.MOE_ERR_INVALID_ARG), (dict(logits_ld=7), nat.MOE_ERR_INVALID_ARG),
    (dict(dlogits_ld=-8), nat.MOE_ERR_INVALID_ARG), (dict(n_experts=513), nat.MOE_ERR_UNSUPPORTED),
    (dict(top_k=17, n_experts=64), nat.MOE_ERR_UNSUPPORTED), (dict(T=1 << 28), nat.MOE_ERR_UNSUPPORTED),
    (dict(n_seqs=(1 << 20) + 1), nat.MOE_ERR_UNSUPPORTED)])
def test_bad_configurations_are_refused(bad, status):
    cfg = nat.balance_config(**{**dict(T=64, n_experts=8, top_k=2, n_seqs=3), **bad})
    assert nat.moe_balance_workspace_bytes(cfg) == 0
    assert _loss(cfg) == status and _grad(cfg) == status


def test_bad_pointers_are_refused():
    cfg = nat.balance_config(64, 8, 2, 3)
    for name in ("logits", "idx", "seqs", "loss", "counts", "tokens"):
        assert _loss(cfg, **{name: None}) == nat.MOE_ERR_INVALID_ARG, name
        assert _loss(cfg, **{name: MIS}) == nat.MOE_ERR_INVALID_ARG, name
    for name in ("mask", "P_"):
        assert _loss(cfg, **{name: MIS}) == nat.MOE_ERR_INVALID_ARG, name
    for name in ("logits", "seqs", "counts", "tokens", "dlogits"):
        assert _grad(cfg, **{name: None}) == nat.MOE_ERR_INVALID_ARG, name
        assert _grad(cfg, **{name: MIS}) == nat.MOE_ERR_INVALID_ARG, name
    for name in ("mask", "dloss"):
        assert _grad(cfg, **{name: MIS}) == nat.MOE_ERR_INVALID_ARG, name
    assert _grad(cfg, accumulate=2) == nat.MOE_ERR_INVALID_ARG
    need = nat.moe_balance_workspace_bytes(cfg)
    assert _loss(cfg, ws=None) == nat.MOE_ERR_WORKSPACE and _loss(cfg, ws=MIS) == nat.MOE_ERR_WORKSPACE
    assert _loss(cfg, nbytes=need - 1) == nat.MOE_ERR_WORKSPACE
    bad = nat.balance_config(64, 8, 2, 3)
    bad.dtype = 2
    assert _loss(bad) == nat.MOE_ERR_INVALID_ARG


def test_router_entry_points_refuse_missing_arrays():
    lib, cfg = nat.lib(), nat.config(64, 128, 256, 8, 1, 8)
    c, ws = ctypes.byref(cfg), nat.moe_workspace_bytes(cfg)
    assert lib.moe_route_logits(c, OK, OK, None, OK, OK, None, None, *[None] * 4, OK, ws, None) == nat.MOE_ERR_INVALID_ARG
    assert lib.moe_route_logits(c, OK, OK, None, OK, OK, None, MIS, *[None] * 4, OK, ws, None) == nat.MOE_ERR_INVALID_ARG
    assert lib.moe_route_logits(c, OK, OK, None, OK, OK, None, OK, *[None] * 4, OK, ws - 1, None) == nat.MOE_ERR_WORKSPACE
    assert lib.moe_router_backward_dh(c, OK, OK, None, OK, OK, OK, OK, ws, None) == nat.MOE_ERR_INVALID_ARG
    assert lib.moe_router_backward_dh(c, None, OK, OK, OK, OK, OK, OK, ws, None) == nat.MOE_ERR_INVALID_ARG
    assert lib.moe_router_backward_dh(c, OK, OK, OK, OK, OK, OK, OK, ws - 1, None) == nat.MOE_ERR_WORKSPACE
