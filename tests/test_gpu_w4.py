"""4-bit weights through the C ABI: quantisation bit for bit against exact
arithmetic, the expert FFN against fp64 within the bound derived in w4_ref, and
the layer's forward on them.  Needs a B200."""
import numpy as np
import pytest

import oracle
import w4_ref
from mixture_experts_sparse_b200 import inputs
from mixture_experts_sparse_b200 import native as nat
from mixture_experts_sparse_b200.layer import to_device

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)


def _quantize(w, group):
    """[mats, rows, K] tensor -> (q, scale, values back in w's type, values in fp32)"""
    M, R, K = w.shape
    dt = "bf16" if w.dtype == torch.bfloat16 else "f32"
    q = torch.full((M, R, nat.moe_w4_row_bytes(K)), 0xEE, dtype=torch.uint8, device="cuda")
    s = torch.full((M, (K + group - 1) // group, R), -1.0, dtype=torch.bfloat16, device="cuda")
    back, back32 = torch.empty_like(w), torch.empty(w.shape, device="cuda")
    nat.check(nat.moe_quantize_w4(M, R, K, group, dt, w, q, s))
    nat.check(nat.moe_dequantize_w4(M, R, K, group, dt, q, s, back))
    nat.check(nat.moe_dequantize_w4(M, R, K, group, "f32", q, s, back32))
    torch.cuda.synchronize()
    return q, s, back, back32


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,R,K", [(1, 1, 16), (2, 17, 128), (3, 33, 144), (1, 40, 1040), (2, 5, 2064), (1, 130, 512)])
def test_quantisation_is_exact(M, R, K, group, dtype):
    g = torch.Generator().manual_seed(M * R + K + group)
    w = (torch.randn(M, R, K, generator=g) * 0.03).to(dtype)
    w[0, 0, : K // 2] = 0                      # a group of zeros where the group is short enough
    q, s, back, back32 = _quantize(w.cuda(), group)
    for m in range(M):
        qr, sr = w4_ref.quantize(w[m].double().numpy(), group)
        np.testing.assert_array_equal(s[m].double().cpu().numpy(), sr)
        np.testing.assert_array_equal(q[m].cpu().numpy(), w4_ref.pack(qr))
        val = w4_ref.values(qr, sr, group)
        np.testing.assert_array_equal(back32[m].double().cpu().numpy(), val)
        want = torch.from_numpy(val).float().to(dtype)   # exact in fp32, so one rounding
        assert torch.equal(back[m].cpu(), want)


def test_quantisation_ties_and_near_ties():
    # multiples of half a scale, and their fp32 neighbours, must not depend on the quotient's rounding
    s = np.float32(0.01171875 * 1.0078125)
    half = (np.arange(-14, 15) * 0.5).astype(np.float64) * s
    w = np.zeros((3, 128), np.float32)
    w[:, :29] = half
    w[1, :29] = np.nextafter(w[1, :29], np.float32(np.inf))
    w[2, :29] = np.nextafter(w[2, :29], np.float32(-np.inf))
    # scales whose bf16 rounding is a near tie
    m = np.arange(1, 129, dtype=np.float32)
    w2 = np.zeros((256, 128), np.float32)
    w2[:128, 0] = np.float32(7) * (1 + (2 * m + 1) / 512).astype(np.float32)
    w2[128:, 0] = np.nextafter(w2[:128, 0], np.float32(np.inf))
    for a in (w, w2):
        q, sc, _, _ = _quantize(torch.from_numpy(a)[None].cuda(), 128)
        qr, sr = w4_ref.quantize(a.astype(np.float64), 128)
        np.testing.assert_array_equal(sc[0].double().cpu().numpy(), sr)
        np.testing.assert_array_equal(q[0].cpu().numpy(), w4_ref.pack(qr))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantisation_of_extreme_magnitudes(dtype):
    # from the largest to the smallest scales; the reference's bf16 is that of normal numbers, so
    # groups whose scale is subnormal are held to the definition by their codes' range and value only
    g = torch.Generator().manual_seed(9)
    w = torch.randn(1, 40, 128, generator=g)
    w = (w * torch.logspace(-36.5, 37.5, 40, dtype=torch.float64)[None, :, None].float()).to(dtype)
    q, s, _, back = _quantize(w.cuda(), 128)
    qr, sr = w4_ref.quantize(w[0].double().numpy(), 128)
    np.testing.assert_array_equal(s[0].double().cpu().numpy(), sr)
    np.testing.assert_array_equal(q[0].cpu().numpy(), w4_ref.pack(qr))
    tiny = (torch.randn(1, 30, 64, generator=g).double() * torch.logspace(-45, -37.5, 30, dtype=torch.float64)[None, :, None]).to(dtype)
    q, s, _, back = _quantize(tiny.cuda(), 64)
    codes = q.cpu().numpy()
    assert ((codes & 15) >= 1).all() and ((codes >> 4) >= 1).all()   # -7 .. 7
    sv = s.double().cpu()[0, 0]
    live = sv > 0
    # the nearest of the representable multiples, or the largest of them
    x = tiny[0].double() / sv.clamp(min=1e-300)[:, None]
    want = torch.where(live[:, None], x, torch.zeros_like(x)).clamp(-7, 7)
    got = torch.where(live[:, None], back[0].double().cpu() / sv.clamp(min=1e-300)[:, None], torch.zeros_like(x))
    assert ((got - want).abs() <= 0.5).all() and (back[0].cpu()[~live] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_groups_stand_for_nan(bad):
    w = torch.randn(1, 3, 256)
    w[0, 1, 70] = bad
    _, _, _, back = _quantize(w.cuda(), 64)
    nan = back[0].isnan().cpu()
    want = torch.zeros(3, 256, dtype=torch.bool)
    want[1, 64:128] = True
    assert torch.equal(nan, want)


# ------------------------------------------------------------- expert FFN ----

def make_experts(N, d, dff, group, act, bias, seed=0):
    """Random codes over all 16 values and positive scales (quantised layers use 1..15)."""
    rng = np.random.default_rng(seed)

    def mat(rows, K):
        q = rng.integers(-8, 8, (N, rows, K)).astype(np.int8)
        s = w4_ref.bf16(rng.uniform(0.5, 2.0, (N, (K + group - 1) // group, rows)) * 0.3 / np.sqrt(K) / 4)
        return q, s

    def vec(n):
        return w4_ref.bf16(rng.standard_normal((N, n)) * 0.1) if bias else None

    W = dict(w1=mat(dff, d), w3=mat(dff, d) if act == "swiglu" else None, w2=mat(d, dff), b1=vec(dff),
             b3=vec(dff) if act == "swiglu" else None, b2=vec(d))
    dev = {}
    for n in ("w1", "w3", "w2"):
        dev[n] = (None, None) if W[n] is None else (torch.from_numpy(w4_ref.pack(W[n][0])).cuda(),
                                                    torch.from_numpy(W[n][1]).to(torch.bfloat16).cuda())
    for n in ("b1", "b3", "b2"):
        dev[n] = None if W[n] is None else torch.from_numpy(W[n]).to(torch.bfloat16).cuda()
    return W, dev


def weight_args(dev):
    return (*dev["w1"], dev["b1"], *dev["w3"], dev["b3"], *dev["w2"], dev["b2"])


def make_rows(R, d, seed=0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((R, d)).astype(np.float32)).to(torch.bfloat16)


def expert_values(W, e, group):
    return [None if W[n] is None else w4_ref.values(W[n][0][e].astype(np.float64), W[n][1][e], group) for n in ("w1", "w3", "w2")]


def run_ffn(dev, x, offsets, N, d, dff, group, act, R_cap, ws=None, stream=None):
    cfg = nat.config(R_cap, d, dff, N, 1, R_cap, "bf16", act)   # room for R_cap rows
    ws = nat.new_w4_workspace(cfg) if ws is None else ws
    y = torch.full((R_cap, d), 55.0, dtype=torch.bfloat16, device="cuda")
    xe = torch.full((R_cap, d), float("nan"), dtype=torch.bfloat16, device="cuda")   # rows past the last one
    xe[: x.shape[0]] = x.cuda()
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    nat.check(nat.moe_expert_ffn_w4(cfg, group, xe, off, *weight_args(dev), y, ws, stream))
    torch.cuda.synchronize()
    nat.check(nat.moe_read_device_status(ws))
    return y.cpu()


H_STEP = 2.0 ** -8   # H in bf16 (many rows); few rows keep 16 bits, which is only better


def check_ffn(W, x, y, offsets, group, act, rows=None):
    xv = x.double().numpy()
    for e in range(len(offsets) - 1):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            continue
        w1, w3, w2 = expert_values(W, e, group)
        pick = np.arange(a, b) if rows is None else np.unique(np.linspace(a, b - 1, min(rows, b - a)).astype(int))
        bias = [None if W[n] is None else W[n][e] for n in ("b1", "b3", "b2")]
        want, bound = w4_ref.ffn(xv[pick], w1, w3, w2, *bias, act, H_STEP)
        got = y.double().numpy()[pick]
        err = np.abs(got - want)
        assert (err <= bound).all(), f"expert {e}: {np.max(err / bound):.2f} of the bound"
        # far tighter than the worst case: two roundings to bf16 (2^-9 / sqrt 3 each, relative RMS) and spare
        rms = np.sqrt((err ** 2).mean() / (want ** 2).mean())
        assert rms < 3.5e-3, f"expert {e}: relative RMS {rms:.2e}"
    assert (y[offsets[-1]:] == 55).all(), "rows behind the last one were written"


@pytest.mark.parametrize("act", ["relu", "swiglu"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("d,dff,rows,bias", [
    (16, 16, [1], True), (128, 256, [0, 1, 0, 2, 8], False), (144, 208, [9, 0, 16, 17, 3], True),
    (528, 1360, [1, 33, 7, 0], True), (1040, 272, [31, 32, 40, 5], False), (256, 2064, [100, 0, 1], True)])
def test_expert_ffn(d, dff, rows, bias, group, act):
    N, off = len(rows), np.concatenate([[0], np.cumsum(rows)]).tolist()
    W, dev = make_experts(N, d, dff, group, act, bias, seed=d + group)
    x = make_rows(off[-1], d)
    y = run_ffn(dev, x, off, N, d, dff, group, act, off[-1] + 3)
    check_ffn(W, x, y, off, group, act)
    assert torch.equal(y, run_ffn(dev, x, off, N, d, dff, group, act, off[-1] + 3)), "two runs differ"


@pytest.mark.parametrize("act,group,d,dff,rows", [
    ("swiglu", 128, 512, 896, [200, 0, 64, 129, 1, 256]), ("relu", 32, 384, 640, [300, 65, 130]),
    ("swiglu", 64, 272, 528, [128, 127, 66]), ("swiglu", 128, 208, 144, [192, 193, 208, 0, 384, 385, 321]),
    ("relu", 64, 64, 272, [383, 96, 97, 224, 16]), ("relu", 32, 144, 2064, [260, 800]), ("relu", 128, 1024, 272, [513, 2]), ("swiglu", 32, 160, 144, [257, 70])])
def test_expert_ffn_many_rows(act, group, d, dff, rows):
    N, off = len(rows), np.concatenate([[0], np.cumsum(rows)]).tolist()
    W, dev = make_experts(N, d, dff, group, act, True, seed=d)
    x = make_rows(off[-1], d)
    y = run_ffn(dev, x, off, N, d, dff, group, act, off[-1] + 40)
    check_ffn(W, x, y, off, group, act)
    assert torch.equal(y, run_ffn(dev, x, off, N, d, dff, group, act, off[-1] + 40)), "two runs differ"


@pytest.mark.parametrize("act,group", [("swiglu", 128), ("relu", 64), ("swiglu", 32)])
@pytest.mark.parametrize("rows", [[200, 216], [150, 170], [0, 440]])
def test_many_rows_over_a_long_k(act, group, rows):
    # K of more blocks than any ring of barriers is long, ending in the first half of a block (stage 1)
    # and in the second (stage 2); 228 rows an expert on average are a tile of up to 256, 180 one of up to 192
    N, d, dff, off = 2, 3216, 2640, [0, rows[0], sum(rows)]
    W, dev = make_experts(N, d, dff, group, act, False, seed=group)
    x = make_rows(off[-1], d)
    y = run_ffn(dev, x, off, N, d, dff, group, act, off[-1] + 40)
    check_ffn(W, x, y, off, group, act, rows=24)


@pytest.mark.parametrize("act,group", [("relu", 128), ("swiglu", 32)])
@pytest.mark.parametrize("N,d,dff,most", [
    (1, 128, 128, 16), (1, 128, 128, 17), (1, 16, 16, 40), (1, 48, 272, 193), (2, 272, 16, 33), (128, 64, 48, 5), (128, 16, 144, 40)])
def test_expert_ffn_at_the_edges(N, d, dff, most, act, group):
    # one expert and 128, both sides of the rows that decide between the kernels, K of a single block
    rng = np.random.default_rng(d + most)
    rows = rng.integers(0, most + 1, N)
    rows[-1] = most
    off = np.concatenate([[0], np.cumsum(rows)]).tolist()
    W, dev = make_experts(N, d, dff, group, act, True, seed=d)
    x = make_rows(off[-1], d)
    y = run_ffn(dev, x, off, N, d, dff, group, act, off[-1])
    check_ffn(W, x, y, off, group, act)


@pytest.mark.parametrize("rows", [[3, 2], [70, 200]])
@pytest.mark.parametrize("act", ["relu", "swiglu"])
def test_magnitudes_far_from_one(act, rows):
    # rows of x and of the weights at very different powers of two (H and y stay within 2^+-100);
    # with SwiGLU a channel of x and two weight rows far above the others
    N, d, dff, group = 2, 256, 320, 64
    W, dev = make_experts(N, d, dff, group, act, False, seed=3)
    rng = np.random.default_rng(4)
    off = np.concatenate([[0], np.cumsum(rows)]).tolist()
    x = make_rows(off[-1], d).double()
    if act == "relu":
        x *= torch.from_numpy(2.0 ** rng.integers(-40, 41, (off[-1], 1)))
        for n in ("w1", "w2"):
            W[n] = (W[n][0], W[n][1] * 2.0 ** rng.integers(-25, 26, (N, 1, W[n][1].shape[2])))
    else:
        x[:, 7] *= 1000
        W["w1"][1][:, :, 3] *= 64
        W["w3"][1][:, :, 5] *= 64
    for n in ("w1", "w3", "w2"):
        if W[n] is not None:
            dev[n] = (dev[n][0], torch.from_numpy(W[n][1]).to(torch.bfloat16).cuda())
    x = x.to(torch.bfloat16)
    y = run_ffn(dev, x, off, N, d, dff, group, act, off[-1])
    check_ffn(W, x, y, off, group, act)


def test_one_workspace_for_both_kinds_of_experts():
    # the layer on bf16 and on 4-bit experts in turn, few and many rows: each gives what it gives alone
    N, d, dff, group = 4, 128, 272, 32
    W, dev = make_experts(N, d, dff, group, "swiglu", False, seed=5)
    wb = [torch.randn(N, *W[n][0].shape[1:], device="cuda").bfloat16() * 0.05 for n in ("w1", "w3", "w2")]
    for T in (5, 400):
        L = inputs.make_layer(T=T, d_model=d, d_ff=16, n_experts=N, top_k=2, dtype="bf16", seed=T)
        cfg = nat.config(T, d, dff, N, 2, T, "bf16", "swiglu")
        x, w_r, b_r = layer_args(L)

        def both(ws_a, ws_b):
            outs = [torch.empty(T, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            nat.check(nat.moe_forward(cfg, x, w_r, b_r, wb[0], None, wb[1], None, wb[2], None, outs[0], ws=ws_a))
            nat.check(nat.moe_forward_w4(cfg, group, x, w_r, b_r, *weight_args(dev), outs[1], ws=ws_b))
            return outs

        want = both(nat.new_workspace(cfg), nat.new_w4_workspace(cfg))
        ws = nat.new_w4_workspace(cfg)
        for _ in range(3):
            for got, ref in zip(both(ws, ws), want):
                assert torch.equal(got, ref)
        nat.check(nat.moe_read_device_status(ws))


@pytest.mark.parametrize("rows", [[3, 2, 4], [40, 30, 60]])
def test_a_workspace_may_have_held_anything(rows):
    # past its header, in either kernel
    N, d, dff, group, R = 3, 512, 1040, 64, sum(rows)
    W, dev = make_experts(N, d, dff, group, "swiglu", True)
    x, offsets = make_rows(R, d), [0, rows[0], rows[0] + rows[1], R]
    want = run_ffn(dev, x, offsets, N, d, dff, group, "swiglu", R)
    for fill in (0xFF, 0x01):
        ws = nat.new_w4_workspace(nat.config(R, d, dff, N, 1, R, "bf16", "swiglu"))
        ws[256:] = fill
        for _ in range(2):
            assert torch.equal(run_ffn(dev, x, offsets, N, d, dff, group, "swiglu", R, ws=ws), want)


def test_a_rows_result_does_not_depend_on_other_experts_rows():
    N, d, dff, group = 3, 256, 320, 64
    W, dev = make_experts(N, d, dff, group, "swiglu", True)
    x = make_rows(12, d)
    base = run_ffn(dev, x, [0, 4, 8, 12], N, d, dff, group, "swiglu", 12)
    x2 = x.clone()
    x2[4:8] = float("nan")
    other = run_ffn(dev, x2, [0, 4, 8, 12], N, d, dff, group, "swiglu", 12)
    assert torch.equal(base[:4], other[:4]) and torch.equal(base[8:], other[8:]) and other[4:8].isnan().all()


@pytest.mark.parametrize("rows", [[3, 2], [200, 60]])
def test_non_finite_rows_stay_in_their_row(rows):
    d, dff, group, R = 256, 384, 128, sum(rows)
    for act in ("relu", "swiglu"):
        W, dev = make_experts(2, d, dff, group, act, False)
        x = make_rows(R, d)
        off = [0, rows[0], R]
        clean = run_ffn(dev, x, off, 2, d, dff, group, act, R)
        x2 = x.clone()
        x2[1, 5] = float("nan")
        x2[R - 1, 7] = float("inf")
        y = run_ffn(dev, x2, off, 2, d, dff, group, act, R)
        keep = [i for i in range(R) if i not in (1, R - 1)]
        assert torch.equal(y[keep], clean[keep])
        assert y[1].isnan().all() and not torch.isfinite(y[R - 1].float()).any()


def test_offsets_beyond_the_rows_are_clamped():
    d, dff, group = 128, 128, 32
    W, dev = make_experts(2, d, dff, group, "relu", False)
    x = make_rows(6, d)
    y = run_ffn(dev, x, [0, 3, 6], 2, d, dff, group, "relu", 6)
    z = run_ffn(dev, x, [-4, 3, 1 << 30], 2, d, dff, group, "relu", 6)
    assert torch.equal(y, z)


def test_replayed_graph_follows_the_offsets():
    N, d, dff, group, R = 4, 256, 512, 64, 96
    W, dev = make_experts(N, d, dff, group, "swiglu", True)
    cfg = nat.config(R, d, dff, N, 1, R, "bf16", "swiglu")
    ws = nat.new_w4_workspace(cfg)
    x = make_rows(R, d)
    xe, y = x.cuda(), torch.full((R, d), 55.0, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()

    def step():
        nat.check(nat.moe_expert_ffn_w4(cfg, group, xe, off, *weight_args(dev), y, ws))

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for o in ([0, 0, 0, 0, 0], [0, 1, 1, 3, 4], [0, 50, 51, 90, 96]):
        y.fill_(55.0)
        off.copy_(torch.tensor(o, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check_ffn(W, x, y.cpu(), o, group, "swiglu")


def test_two_streams_with_a_workspace_each():
    N, d, dff, group = 4, 512, 1024, 128
    W, dev = make_experts(N, d, dff, group, "swiglu", False)
    off = [0, 2, 5, 5, 7]
    xs = [make_rows(7, d, seed=i) for i in range(2)]
    alone = [run_ffn(dev, x, off, N, d, dff, group, "swiglu", 7) for x in xs]
    cfg = nat.config(7, d, dff, N, 1, 7, "bf16", "swiglu")
    ws = [nat.new_w4_workspace(cfg) for _ in xs]
    ys = [torch.zeros(7, d, dtype=torch.bfloat16, device="cuda") for _ in xs]
    xd, o = [x.cuda() for x in xs], torch.tensor(off, dtype=torch.int32, device="cuda")
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            nat.check(nat.moe_expert_ffn_w4(cfg, group, xd[i], o, *weight_args(dev), ys[i], ws[i], st))
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(ys[i].cpu(), alone[i])


# ------------------------------------------------------------------ layer ----

def layer_args(L):
    return to_device(L["x"]), to_device(L["w_r"]), to_device(L["b_r"])


def routing(T, N, k):
    z = dict(device="cuda")
    i32, f64 = torch.int32, torch.float64
    return dict(idx=torch.zeros(T, k, dtype=i32, **z), gate=torch.zeros(T, k, **z), pos=torch.zeros(T, k, dtype=i32, **z),
                drop=torch.zeros(T, k, dtype=torch.uint8, **z), counts=torch.zeros(k, N, dtype=i32, **z),
                kept=torch.zeros(N, dtype=i32, **z), offsets=torch.zeros(N + 1, dtype=i32, **z),
                f=torch.zeros(N, dtype=f64, **z), P=torch.zeros(N, dtype=f64, **z), aux=torch.zeros(1, dtype=f64, **z))


@pytest.mark.parametrize("T,d,dff,N,k,C,act,group,order", [
    (1, 128, 256, 8, 2, 1, "swiglu", 64, 0), (1, 256, 128, 4, 1, 1, "relu", 128, 0),
    (7, 128, 256, 8, 2, 2, "swiglu", 32, 0), (64, 256, 272, 16, 1, 3, "relu", 64, 1),
    (50, 128, 128, 4, 1, 13, "relu", 32, 2), (900, 256, 320, 8, 2, 200, "swiglu", 64, 0), (0, 128, 128, 4, 1, 0, "relu", 32, 0)])
def test_layer_forward(T, d, dff, N, k, C, act, group, order):
    L = inputs.make_layer(T=T, d_model=d, d_ff=16, n_experts=N, top_k=k, dtype="bf16", seed=T + d,
                          router_bias=np.linspace(1.0, 0.0, N).astype(np.float32))
    W, dev = make_experts(N, d, dff, group, act, True, seed=T)
    cfg = nat.config(T, d, dff, N, k, C, "bf16", act, priority=order)
    ws = nat.new_w4_workspace(cfg)
    x, w_r, b_r = layer_args(L)
    r, r2 = routing(T, N, k), routing(T, N, k)
    out = torch.full((max(T, 1), d), float("nan"), dtype=torch.bfloat16, device="cuda")[:T]
    nat.check(nat.moe_forward_w4(cfg, group, x, w_r, b_r, *weight_args(dev), out, **r, ws=ws))
    # the routing is moe_forward's
    wb = [None if W[n] is None else torch.zeros(N, *W[n][0].shape[1:], dtype=torch.bfloat16, device="cuda") for n in ("w1", "w3", "w2")]
    out2 = torch.empty_like(out)
    nat.check(nat.moe_forward(cfg, x, w_r, b_r, wb[0], None, wb[1], None, wb[2], None, out2, **r2, ws=ws))
    torch.cuda.synchronize()
    nat.check(nat.moe_read_device_status(ws))
    for n in r:
        assert torch.equal(r[n], r2[n]), n
    if T == 0:
        return
    # outputs: every kept assignment's expert output times its gate
    xv = torch.from_numpy(oracle.widen(L["x"]))
    idx, gate, drop = r["idx"].cpu().numpy(), r["gate"].double().cpu().numpy(), r["drop"].cpu().numpy()
    want, bound = np.zeros((T, d)), np.zeros((T, d))
    for e in range(N):
        w1, w3, w2 = expert_values(W, e, group)
        for j in range(k):
            t = np.nonzero((idx[:, j] == e) & (drop[:, j] == 0))[0]
            if len(t):
                y, b = w4_ref.ffn(xv.numpy()[t], w1, w3, w2, W["b1"][e], None if W["b3"] is None else W["b3"][e], W["b2"][e], act, H_STEP)
                want[t] += gate[t, j][:, None] * y
                bound[t] += gate[t, j][:, None] * b
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound) + 1e-6 * np.abs(want)).all()
    assert (got[drop.all(axis=1)] == 0).all()


def test_router_training_over_frozen_4bit_experts():
    """The operators as a user runs them together: quantise the experts, route with logits, run the 4-bit
    experts, the balance loss of a padded batch, and the router's gradient from both losses."""
    T, d, dff, N, k, S, group, alpha, zc = 300, 256, 384, 8, 2, 5, 64, 0.05, 0.01
    import balance_ref
    L = inputs.make_layer(T=T, d_model=d, d_ff=dff, n_experts=N, top_k=k, act="swiglu", dtype="bf16", seed=11)
    rng = np.random.default_rng(2)
    mask = (rng.random(T) < 0.8).astype(np.uint8)
    seqs = np.array([0, 40, 40, 150, 260, 290], np.int32)
    x, w_r, b_r = layer_args(L)
    z = dict(device="cuda")
    W, vals = {}, {}
    for n, rows, K in (("w1", dff, d), ("w3", dff, d), ("w2", d, dff)):
        w = to_device(L[n]).view(N, rows, K)
        q, s, _, v32 = _quantize(w, group)
        W[n], vals[n] = (q, s), v32.double().cpu().numpy()
    cfg = nat.config(T, d, dff, N, k, T, "bf16", "swiglu", alpha=0.0)
    ws = nat.new_w4_workspace(cfg)
    r = routing(T, N, k)
    probs, logits = torch.zeros(T, N, **z), torch.zeros(T, N, **z)
    R = T * k
    row_token, row_gate = torch.zeros(R, dtype=torch.int32, **z), torch.zeros(R, **z)
    xe, ye = torch.zeros(R, d, dtype=torch.bfloat16, **z), torch.zeros(R, d, dtype=torch.bfloat16, **z)
    out, dout = torch.zeros(T, d, dtype=torch.bfloat16, **z), make_rows(T, d, seed=9).cuda()
    bc = nat.balance_config(T, N, k, S, "f32", alpha, zc)
    bws = nat.new_balance_workspace(bc)
    loss, cnt, tok = torch.zeros(2, **z), torch.zeros(S, N, dtype=torch.int32, **z), torch.zeros(S + 2, dtype=torch.int32, **z)
    dgate, dh = torch.zeros(T, k, **z), torch.zeros(T, N, **z)
    dw, db, dx = torch.zeros(N, d, **z), torch.zeros(N, **z), torch.zeros(T, d, **z)
    md, sd = to_device(mask), to_device(seqs)
    weights = (*W["w1"], None, *W["w3"], None, *W["w2"], None)

    def step():
        nat.check(nat.moe_route_logits(cfg, x, w_r, b_r, r["idx"], r["gate"], probs, logits, r["f"], r["P"], r["aux"], None, ws))
        nat.check(nat.moe_dispatch(cfg, x, r["idx"], r["gate"], r["pos"], r["drop"], r["counts"], r["kept"], r["offsets"],
                                   row_token, row_gate, xe, ws))
        nat.check(nat.moe_expert_ffn_w4(cfg, group, xe, r["offsets"], *weights, ye, ws))
        nat.check(nat.moe_combine(cfg, ye, r["idx"], r["pos"], r["drop"], r["gate"], r["offsets"], out))
        nat.check(nat.moe_balance_loss(bc, logits, r["idx"], md, sd, loss, cnt, None, tok, bws))
        nat.check(nat.moe_gate_grad(cfg, dout, ye, r["idx"], r["pos"], r["drop"], r["offsets"], dgate))
        nat.check(nat.moe_router_backward(cfg, x, w_r, probs, r["idx"], r["gate"], r["f"], dgate, dh, None, None, None, ws))
        nat.check(nat.moe_balance_loss_backward(bc, logits, md, sd, cnt, tok, None, dh, True))
        nat.check(nat.moe_router_backward_dh(cfg, x, w_r, dh, dw, db, dx, ws))

    step()
    torch.cuda.synchronize()
    whole = torch.zeros_like(out)
    nat.check(nat.moe_forward_w4(cfg, group, x, w_r, b_r, *weights, whole, ws=ws))
    torch.cuda.synchronize()
    assert torch.equal(whole, out)
    # fp64: outputs, losses, gradient
    xv, idx, gate = oracle.widen(L["x"]), r["idx"].cpu().numpy(), r["gate"].double().cpu().numpy()
    y64, b64 = np.zeros((T, k, d)), np.zeros((T, k, d))
    for e in range(N):
        t, j = np.nonzero(idx == e)
        if len(t):
            y64[t, j], b64[t, j] = w4_ref.ffn(xv[t], vals["w1"][e], vals["w3"][e], vals["w2"][e], None, None, None, "swiglu", H_STEP)
    want, bound = (gate[..., None] * y64).sum(1), (gate[..., None] * b64).sum(1)
    assert (np.abs(out.double().cpu().numpy() - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound) + 1e-6 * np.abs(want)).all()
    hv = logits.double().cpu().numpy()
    ref, counts, _, _ = balance_ref.loss(hv, idx, mask, seqs, alpha, zc)
    np.testing.assert_array_equal(cnt.cpu().numpy(), counts)
    np.testing.assert_allclose(loss.cpu().numpy(), ref, rtol=2.0 ** -14)
    dg = (dout.double().cpu().numpy()[:, None, :] * y64).sum(-1)
    gb = (np.abs(dout.double().cpu().numpy())[:, None, :] * b64).sum(-1) + 2.0 ** -14 * np.abs(dg)
    assert (np.abs(dgate.double().cpu().numpy() - dg) <= gb).all()
    gp = gate[:, 0] * gate[:, 1] * (dgate.double().cpu().numpy()[:, 0] - dgate.double().cpu().numpy()[:, 1])
    path = np.zeros((T, N))
    path[np.arange(T), idx[:, 0]] += gp
    path[np.arange(T), idx[:, 1]] -= gp
    g, _, _ = balance_ref.gradient(hv, k, mask, seqs, alpha, zc, counts)
    total = path + g
    for got, val in ((dh, total), (dw, total.T @ xv), (db, total.sum(0)), (dx, total @ L["w_r"].astype(np.float64))):
        # the router backward's tolerance on its own inputs: 1e-5 of the largest magnitude
        assert np.abs(got.double().cpu().numpy() - val).max() <= 1e-5 * np.abs(val).max()
    # captured and replayed: the same bits
    first = [t.clone() for t in (out, loss, cnt, dh, dw, db, dx)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (out, loss, cnt, dh, dw, db, dx):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, (out, loss, cnt, dh, dw, db, dx)):
        assert torch.equal(a, b)
