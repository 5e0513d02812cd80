"""Balance loss, counts and gradient through the C ABI against their fp64
definition (balance_ref).

Error bounds.  p: the difference h - max is rounded once (2^-24 |h - max|
absolute, hence relative in p; |h - max| < 24 in these inputs), exp is good to
2^-22, the row sum adds up to 17 fp32 additions per lane and tree (2^-24 each)
and the division one rounding: below 24 2^-24 + 4 2^-24 + 18 2^-24 < 2^-18
relative.  Sums of p are of one sign, with at most a few hundred fp32
additions per lane before fp64: 2^-18 + 256 2^-24 < 2^-15 in the worst case; the
gradient's error is at most 2^-17 of the sum of its terms' magnitudes (p's
bound and as much again for the dot product and lse) plus the rounding to its
type."""
import numpy as np
import pytest

import balance_ref
import oracle
from mixture_experts_sparse_b200 import inputs
from mixture_experts_sparse_b200 import native as nat
from mixture_experts_sparse_b200.layer import to_device

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

TOL_P, TOL_GRAD = 2.0 ** -15, 2.0 ** -17
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _seqs(T, S, rng, tail):
    cuts = np.sort(rng.integers(0, T - tail + 1, S - 1))
    return np.concatenate([[0], cuts, [T - tail]]).astype(np.int32)


def make(T, N, k, S, dtype, seed=0, mask=True, tail=0, head=0):
    rng = np.random.default_rng(seed)
    h = torch.from_numpy(rng.standard_normal((T, N)).astype(np.float32) * 2)
    h = h.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    idx = np.argsort(-h.double().numpy(), axis=1, kind="stable")[:, :k].astype(np.int32)
    seqs = _seqs(T, S, rng, tail)
    seqs[0] = min(head, seqs[1])
    return h, idx, seqs, (rng.random(T) < 0.75).astype(np.uint8) if mask else None


def strided(h, ld):
    """The same rows in a wider buffer whose other columns hold NaN."""
    if ld == 0:
        return h.cuda()
    wide = torch.full((h.shape[0], ld), float("nan"), dtype=h.dtype)
    wide[:, :h.shape[1]] = h
    return wide.cuda()


def run(h, idx, seqs, mask, dtype, alpha=0.3, zc=0.2, g=None, ld=0, dld=0, accumulate=None, ws=None, stream=None):
    T, N = h.shape
    k, S = idx.shape[1], (1 if seqs is None else len(seqs) - 1)
    cfg = nat.balance_config(T, N, k, S, dtype, alpha, zc, ld, dld)
    ws = nat.new_balance_workspace(cfg) if ws is None else ws
    dev = dict(device="cuda")
    o = dict(loss=torch.full((2,), np.nan, **dev), counts=torch.full((S, N), -7, dtype=torch.int32, **dev),
             P=torch.full((S, N), np.nan, **dev), tokens=torch.full((S + 2,), -7, dtype=torch.int32, **dev))
    hd, sd, md = strided(h, ld), to_device(seqs), to_device(mask)
    nat.check(nat.moe_balance_loss(cfg, hd, to_device(idx), md, sd, o["loss"], o["counts"], o["P"], o["tokens"], ws,
                                   stream))
    d = torch.full((T, dld or N), 77.0, dtype=h.dtype, **dev)
    if accumulate is not None:
        d[:, :N] = accumulate
    gd = None if g is None else torch.tensor(g, dtype=torch.float32, **dev)
    nat.check(nat.moe_balance_loss_backward(cfg, hd, md, sd, o["counts"], o["tokens"], gd, d, accumulate is not None,
                                            stream))
    torch.cuda.synchronize()
    o["d"] = d
    return {q: v.cpu() for q, v in o.items()}


def check(h, idx, seqs, mask, dtype, o, alpha=0.3, zc=0.2, g=(1.0, 1.0), add=None):
    hv = h.double().numpy()
    T, N = hv.shape
    ref, counts, P, tokens = balance_ref.loss(hv, idx, mask, seqs, alpha, zc)
    np.testing.assert_array_equal(o["counts"].numpy(), counts)
    np.testing.assert_array_equal(o["tokens"].numpy(), tokens)
    np.testing.assert_allclose(o["P"].numpy(), P, rtol=TOL_P, atol=1e-30)
    np.testing.assert_allclose(o["loss"].numpy(), ref, rtol=2 * TOL_P, atol=1e-30)
    d, size, written = balance_ref.gradient(hv, idx.shape[1], mask, seqs, alpha, zc, counts, g)
    got = o["d"].double().numpy()
    assert (got[:, N:] == 77).all(), "columns past N were written"
    base = np.zeros((T, N)) if add is None else add.double().numpy()
    want = d + base
    assert (got[~written, :N] == (77 if add is None else base[~written])).all(), "rows of no sequence were written"
    err = np.abs(got[:, :N] - want)[written]
    bound = (TOL_GRAD * size + HALF_STEP[dtype] * (np.abs(want) + TOL_GRAD * size))[written] + 1e-37
    assert (err <= bound).all(), f"worst {np.max(err / bound):.2f} of the bound"


@pytest.mark.parametrize("T,N,k,S,dtype,mask,tail", [
    (1, 1, 1, 1, "f32", False, 0), (1, 4, 4, 1, "bf16", False, 0), (2, 3, 2, 2, "f32", True, 0),
    (63, 5, 2, 1, "f32", False, 0), (64, 8, 2, 3, "bf16", True, 0), (65, 8, 1, 65, "f32", False, 0),
    (129, 9, 3, 4, "bf16", True, 7), (1000, 16, 2, 11, "f32", True, 0), (1000, 17, 1, 3, "bf16", False, 1),
    (777, 32, 4, 300, "f32", True, 0), (2049, 33, 2, 5, "f32", True, 64), (4097, 60, 4, 37, "bf16", True, 91),
    (3000, 64, 1, 6, "f32", False, 0), (1500, 127, 8, 2, "bf16", True, 0), (2500, 128, 2, 9, "f32", True, 5),
    (900, 129, 16, 3, "f32", True, 0), (1300, 255, 6, 4, "bf16", True, 0), (1300, 256, 8, 4, "f32", True, 0),
    (700, 257, 3, 2, "bf16", False, 0), (515, 511, 2, 3, "f32", True, 3), (515, 512, 16, 3, "bf16", True, 0),
    (40000, 8, 2, 1, "f32", False, 0), (30011, 64, 2, 130, "bf16", True, 11)])
def test_matches_definition(T, N, k, S, dtype, mask, tail):
    h, idx, seqs, m = make(T, N, k, S, dtype, seed=T + N, mask=mask, tail=tail)
    o = run(h, idx, seqs, m, dtype)
    check(h, idx, seqs, m, dtype, o)
    again = run(h, idx, seqs, m, dtype)
    for q in o:
        assert torch.equal(o[q], again[q]), f"{q} differs between two runs"


@pytest.mark.parametrize("T,N,k,S,mask", [
    (1, 512, 16, 1, False), (3000, 8, 8, 3, True), (4096, 32, 16, 4, True), (5000, 4, 4, 2, False), (20000, 128, 3, 1, True),
    (9000, 16, 16, 2, True), (3000, 16, 2, 3000, False), (260, 200, 5, 260, True), (100000, 256, 8, 1, True)])
def test_tiles_batches_and_units(T, N, k, S, mask):
    # several tiles summed by the last of them, more choices than are loaded ahead, sequences of a row
    # or none that cut every batch, one sequence over all tiles
    h, idx, seqs, m = make(T, N, k, S, "f32", seed=T, mask=mask)
    for _ in range(2):
        check(h, idx, seqs, m, "f32", run(h, idx, seqs, m, "f32"))


def test_one_group_without_offsets():
    h, idx, _, _ = make(999, 24, 3, 1, "f32", mask=False)
    o = run(h, idx, None, None, "f32")
    check(h, idx, None, None, "f32", o)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,ld,dld", [(8, 12, 0), (8, 11, 20), (60, 64, 61), (130, 0, 256)])
def test_strided_rows(N, ld, dld, dtype):
    h, idx, seqs, m = make(300, N, 2, 4, dtype)
    check(h, idx, seqs, m, dtype, run(h, idx, seqs, m, dtype, ld=ld, dld=dld))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_upstream_gradients_and_accumulation(dtype):
    h, idx, seqs, m = make(501, 20, 2, 4, dtype, tail=9, head=6)
    g = (-0.7, 2.5)
    check(h, idx, seqs, m, dtype, run(h, idx, seqs, m, dtype, g=g), g=g)
    add = (torch.randn(501, 20) * 1e-3).to(h.dtype)
    o = run(h, idx, seqs, m, dtype, g=g, accumulate=add.cuda())
    check(h, idx, seqs, m, dtype, o, g=g, add=add)
    keep = torch.from_numpy(m == 0)
    assert torch.equal(o["d"][keep], add[keep])   # masked rows are not touched


def test_gradient_matches_differences_of_the_kernels_own_loss():
    # steps of 1/16: truncation h^2 / 6 = 6.6e-4 times the third derivative (alpha N + a few
    # z_coef lse: below 3 here), rounding 2 TOL_P |loss| / (2 h) with |loss| < 2
    h, idx, seqs, m = make(6, 4, 2, 2, "f32", mask=False)
    o = run(h, idx, seqs, m, "f32")
    for t in range(6):
        for j in range(4):
            v = []
            for sgn in (1, -1):
                x = h.clone()
                x[t, j] += sgn * 0.0625
                v.append(run(x, idx, seqs, m, "f32")["loss"].double().sum().item())
            assert abs((v[0] - v[1]) / 0.125 - o["d"][t, j].item()) < 2e-3 + 2 * TOL_P * 2 / 0.125


def test_padding_cannot_leak():
    # masked rows may hold anything; -inf logits are experts that cannot be chosen
    h, idx, seqs, m = make(400, 12, 2, 3, "f32")
    h[:, 5] = float("-inf")
    h[10] = float("-inf")
    m[10] = 1
    idx[7] = (-1, 12)          # choices outside [0, N) are not counted
    clean = run(h, idx, seqs, m, "f32")
    check(h, idx, seqs, m, "f32", clean)
    off = torch.from_numpy(m == 0)
    for junk in (float("nan"), float("inf"), float("-inf"), torch.finfo(torch.float32).min):
        x, i = h.clone(), idx.copy()
        x[off] = junk
        i[m == 0] = 1 << 30
        o = run(x, i, seqs, m, "f32")
        for q in o:
            assert torch.equal(o[q], clean[q]), (junk, q)
    low = h.clone()
    low[:, 5] = torch.finfo(torch.float32).min   # the type's lowest value masks an expert as -inf does
    low[10] = h[10]
    o = run(low, idx, seqs, m, "f32")
    for q in ("loss", "counts", "P"):
        assert torch.equal(o[q], clean[q]), q


def test_nan_logits_make_their_sequence_nan_only():
    h, idx, seqs, m = make(300, 8, 1, 3, "f32", mask=False)
    t = int(seqs[1])
    h[t, 3] = float("nan")
    o = run(h, idx, seqs, m, "f32")
    P, s = o["P"], int(np.searchsorted(seqs, t, side="right")) - 1
    assert P[s].isnan().all() and not P[[i for i in range(3) if i != s]].isnan().any()
    assert o["d"][t].isnan().all() and not o["d"][t - 1].isnan().any()


@pytest.mark.parametrize("T", [0, 1, 130])
def test_nothing_to_count(T):
    h, idx = torch.zeros(T, 6), np.zeros((T, 2), np.int32)
    seqs = np.array([0, 0, T, T], np.int32)
    o = run(h, idx, seqs, np.zeros(T, np.uint8), "f32")
    assert (o["loss"] == 0).all() and (o["counts"] == 0).all() and (o["P"] == 0).all() and (o["tokens"] == 0).all()
    assert (o["d"] == 0).all()


def test_offsets_are_clamped():
    h, idx, _, _ = make(200, 8, 2, 2, "f32", mask=False)
    o = run(h, idx, np.array([-5, 90, 1 << 30], np.int32), None, "f32")
    check(h, idx, np.array([0, 90, 200], np.int32), None, "f32", o)


def test_replayed_graph_on_a_side_stream():
    h, idx, seqs, m = make(3000, 64, 2, 7, "f32")
    cfg = nat.balance_config(3000, 64, 2, 7, "f32", 0.3, 0.2)
    ws = nat.new_balance_workspace(cfg)
    hd, idxd, sd, md = h.cuda(), to_device(idx), to_device(seqs), to_device(m)
    loss, counts = torch.zeros(2, device="cuda"), torch.zeros(7, 64, dtype=torch.int32, device="cuda")
    P, tokens, d = torch.zeros(7, 64, device="cuda"), torch.zeros(9, dtype=torch.int32, device="cuda"), torch.zeros_like(hd)
    side = torch.cuda.Stream()

    def step():
        nat.check(nat.moe_balance_loss(cfg, hd, idxd, md, sd, loss, counts, P, tokens, ws))
        nat.check(nat.moe_balance_loss_backward(cfg, hd, md, sd, counts, tokens, None, d, False))

    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for seed in (1, 2):
        h2, idx2, _, _ = make(3000, 64, 2, 7, "f32", seed=seed)
        hd.copy_(h2)
        idxd.copy_(to_device(idx2))
        graph.replay()
        torch.cuda.synchronize()
        check(h2, idx2, seqs, m, "f32", dict(loss=loss.cpu(), counts=counts.cpu(), P=P.cpu(), tokens=tokens.cpu(), d=d.cpu()))


@pytest.mark.parametrize("T,d,N,k,dtype", [(3000, 128, 8, 1, "bf16"), (2049, 256, 64, 2, "bf16"), (500, 128, 128, 2, "bf16"),
                                           (777, 64, 40, 2, "f32"), (130, 64, 8, 1, "f32"), (1, 64, 12, 1, "f32")])
def test_router_logits(T, d, N, k, dtype):
    # the other outputs are moe_route_z's bits; softmax of the logits is probs, and the
    # balance loss of one group is aux (first choices) and the z-loss
    L = inputs.make_layer(T=T, d_model=d, d_ff=64, n_experts=N, top_k=k, dtype=dtype, seed=T,
                          router_bias=np.linspace(0.4, 0.0, N).astype(np.float32))
    cfg = nat.config(T, d, 64, N, k, T, dtype, "relu")
    ws = nat.new_workspace(cfg)
    x, w, b = to_device(L["x"]), to_device(L["w_r"]), to_device(L["b_r"])

    def outs():
        z = dict(device="cuda")
        return [torch.zeros(T, k, dtype=torch.int32, **z), torch.zeros(T, k, **z), torch.zeros(T, N, **z),
                torch.zeros(N, dtype=torch.float64, **z), torch.zeros(N, dtype=torch.float64, **z),
                torch.zeros(1, dtype=torch.float64, **z), torch.zeros(1, dtype=torch.float64, **z)]

    a, c = outs(), outs()
    logits = torch.full((T, N), np.nan, device="cuda")
    nat.check(nat.moe_route_z(cfg, x, w, b, *a, ws))
    nat.check(nat.moe_route_logits(cfg, x, w, b, *c[:3], logits, *c[3:], ws))
    torch.cuda.synchronize()
    for p, q in zip(a, c):
        assert torch.equal(p, q)
    ref = oracle.widen(L["x"]) @ L["w_r"].astype(np.float64).T + L["b_r"]
    # fp32 accumulation of d products of magnitude |x w|
    size = np.abs(oracle.widen(L["x"])) @ np.abs(L["w_r"]).astype(np.float64).T + np.abs(L["b_r"])
    assert (np.abs(logits.cpu().numpy() - ref) <= 2.0 ** -20 * size + 1e-7).all()
    first = c[0][:, :1].contiguous()
    o = run(logits.cpu(), first.cpu().numpy(), None, None, "f32", alpha=1e-2, zc=1.0)
    np.testing.assert_allclose(o["loss"].numpy(), [c[5].item(), c[6].item()], rtol=1e-5)


def test_router_gradient_of_the_balance_loss():
    # router logits -> loss -> gradient on top of the gate path -> dW_r, db_r, dx
    T, d, N, k, alpha, zc = 1200, 128, 16, 2, 0.05, 0.01
    L = inputs.make_layer(T=T, d_model=d, d_ff=64, n_experts=N, top_k=k, dtype="bf16", seed=3,
                          router_bias=np.linspace(0.4, 0.0, N).astype(np.float32))
    _, _, seqs, mask = make(T, N, k, 5, "f32", seed=4)
    cfg = nat.config(T, d, 64, N, k, T, "bf16", "relu", alpha=0.0)
    ws = nat.new_workspace(cfg)
    x, w, b = to_device(L["x"]), to_device(L["w_r"]), to_device(L["b_r"])
    z = dict(device="cuda")
    idx, gate, probs = torch.zeros(T, k, dtype=torch.int32, **z), torch.zeros(T, k, **z), torch.zeros(T, N, **z)
    logits, f = torch.zeros(T, N, **z), torch.zeros(N, dtype=torch.float64, **z)
    nat.check(nat.moe_route_logits(cfg, x, w, b, idx, gate, probs, logits, f, None, None, None, ws))
    bc = nat.balance_config(T, N, k, 5, "f32", alpha, zc)
    bws = nat.new_balance_workspace(bc)
    loss, counts = torch.zeros(2, **z), torch.zeros(5, N, dtype=torch.int32, **z)
    tokens = torch.zeros(7, dtype=torch.int32, **z)
    sd, md = to_device(seqs), to_device(mask)
    nat.check(nat.moe_balance_loss(bc, logits, idx, md, sd, loss, counts, None, tokens, bws))
    dgate = torch.from_numpy(np.random.default_rng(5).standard_normal((T, k)).astype(np.float32)).cuda()
    dh = torch.zeros(T, N, **z)
    nat.check(nat.moe_router_backward(cfg, x, w, probs, idx, gate, f, dgate, dh, None, None, None, ws))
    nat.check(nat.moe_balance_loss_backward(bc, logits, md, sd, counts, tokens, None, dh, True))
    dw, db, dx = torch.zeros(N, d, **z), torch.zeros(N, **z), torch.zeros(T, d, **z)
    nat.check(nat.moe_router_backward_dh(cfg, x, w, dh, dw, db, dx, ws))
    torch.cuda.synchronize()
    nat.check(nat.moe_read_device_status(ws))
    ref = oracle.router_backward(L["x"], L["w_r"], probs.cpu().numpy(), idx.cpu().numpy(), gate.cpu().numpy(),
                                 f.cpu().numpy(), dgate.cpu().numpy(), 0.0)["dh"].astype(np.float64)
    g, _, _ = balance_ref.gradient(logits.double().cpu().numpy(), k, mask, seqs, alpha, zc, counts.cpu().numpy())
    total = ref + g
    xv = oracle.widen(L["x"])
    for got, want in ((dh, total), (dw, total.T @ xv), (db, total.sum(0)), (dx, total @ L["w_r"].astype(np.float64))):
        # the router backward's own tolerance: 1e-5 of the largest magnitude
        assert np.abs(got.double().cpu().numpy() - want).max() <= 1e-5 * np.abs(want).max()


@pytest.mark.parametrize("N", [1, 2, 3, 4])
@pytest.mark.parametrize("T", [1, 31, 257, 1025, 5000])
def test_counts_of_few_experts_in_one_sequence(T, N):
    # a row per lane and no sequence to look for: a warp's counters are cleared and counted in with
    # no exchange between its lanes but the one that orders the two
    h, idx, _, m = make(T, N, N, 1, "f32", seed=T + N)
    for _ in range(5):
        check(h, idx, None, m, "f32", run(h, idx, None, m, "f32"))


@pytest.mark.parametrize("T,N,dtype", [(2300, 512, "f32"), (1111, 256, "f32"), (1500, 64, "bf16"), (700, 33, "f32")])
def test_sums_of_p_past_a_lane_run_in_64_bits(T, N, dtype):
    # every tile is one row per lane, so no two values of p meet in fp32: P and the loss are one
    # rounding (2^-24) of the fp64 sums of the kernel's own p, which single-row sequences give.
    # Each further rounding of a tile's share to fp32 would be as large.
    h, idx, _, _ = make(T, N, 1, 1, dtype, seed=T, mask=False)
    alone = run(h, idx, np.arange(T + 1, dtype=np.int32), None, dtype)
    p = alone["P"].double().numpy()
    o = run(h, idx, None, None, dtype, alpha=0.25, zc=0.0)
    mean = p.mean(axis=0)
    one = 2.0 ** -24 * (1 + 2.0 ** -20)   # fp64's own rounding: T 2^-53
    assert (np.abs(o["P"].double().numpy()[0] - mean) <= one * mean).all()
    aux = 0.25 * N * (o["counts"].double().numpy()[0] / T * mean).sum()
    assert abs(o["loss"][0].item() - aux) <= one * aux
