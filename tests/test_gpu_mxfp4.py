"""GPU MXFP4: the codec bit for bit against the oracle, and the linear over an
MXFP4 base, forward and backward, within the rounding it does (the derivation
heads test_gpu_dropout.py: the base product's inputs are exact, so only fp32
sums, the bf16 operands H and dH of the adapter and the bf16 outputs round).
"""

import numpy as np
import pytest
import torch

from bit_nf4_quantized_08_amd import lib, synth
from oracle import dropout as D
from oracle import mxfp4 as MX
from tests.gpu_util import REL_FRO_TOL, dev, guarded, guards_intact, host, rel_fro, say, to_dev
from tests.test_gpu_dropout import EPS, HALF, OFF, SEED, check_step

pytestmark = pytest.mark.gpu


def _quantize_guarded(x):
    """Library codes and scales of a device tensor, in guard bands."""
    rows, cols = x.shape
    C = -(-cols // 256)
    fc, codes = guarded(rows * 128 * C, torch.uint8)
    fs, scales = guarded(rows * 8 * C, torch.uint8)
    m = lib.mxfp4_quantize(x, out=lib.MXMatrix(codes.view(rows, 128 * C), scales.view(C, rows, 8), rows, cols))
    assert guards_intact(fc, rows * 128 * C) and guards_intact(fs, rows * 8 * C)
    return m


def _check_codec(x):
    """x: CPU tensor, bf16 or fp32."""
    m = _quantize_guarded(x.to(dev()))
    codes, scales = MX.quantize(x.float().numpy())
    np.testing.assert_array_equal(host(m.codes), codes)
    np.testing.assert_array_equal(host(m.scales), scales)
    want = MX.dequant(codes, scales, x.shape[1])
    for dt, kind in ((torch.float32, "f32"), (torch.bfloat16, "bf16")):
        nb = x.numel() * (4 if kind == "f32" else 2)
        full, out = guarded(nb, dt)
        lib.mxfp4_dequant(m, out=out.view(x.shape))
        assert guards_intact(full, nb)
        np.testing.assert_array_equal(host(out.view(x.shape)).astype(np.float64), want)
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows, cols", [(1, 1), (1, 7), (3, 31), (2, 32), (5, 33), (4, 64), (1, 255), (7, 256), (3, 257),
                                        (65, 520), (33, 1000), (1, 4096), (130, 2051), (1030, 24)])
def test_codec_bit_for_bit(dtype, rows, cols):
    say(f"mxfp4 codec {rows}x{cols} {dtype}")
    x = synth.gaussian((rows, cols), 1.0, rows * 7 + cols) * np.exp(synth.gaussian((rows, 1), 3.0, 5))
    _check_codec(torch.from_numpy(x.astype(np.float32)).to(dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [320, 321])
def test_codec_edge_blocks(dtype, cols):
    """Ties, signs of zero, subnormals, the largest values, infinities and NaN, on the aligned and the ragged path."""
    say(f"mxfp4 edge blocks {dtype} cols={cols}")
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0]
    x = torch.zeros((12, cols))
    for i, u in enumerate((1.0, 2.0 ** -100, 2.0 ** 100, 2.0 ** 125)):
        x[i, :9] = torch.tensor([4.0] + ties) * u
        x[i, 32:41] = -x[i, :9]
    x[4, :4] = torch.tensor([-0.0, 0.0, -0.0, 0.0])
    x[5, :6] = torch.tensor([1e-40, -1e-40, 2.0 ** -126, 2.0 ** -130, 1e-45, -2.0 ** -127])
    x[6, :3] = torch.tensor([2.0 ** -133, -(2.0 ** -133), 0.0])
    x[7, 5], x[7, 40], x[7, 70] = float("inf"), float("-inf"), float("nan")
    x[8, :] = 3.3e38
    x[9, 31], x[9, 32] = 1.0, 1000.0
    x[10, :32] = torch.linspace(-8, 8, 32)
    x[11, cols - 1] = -1.0
    _check_codec(x.to(dtype))


def test_codec_of_very_many_rows():
    """2^29 rows of one column and some (75 GB): the grid and the offsets beyond 32 bits."""
    rows = (1 << 29) + 7
    say(f"codec rows={rows} cols=1")
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    x = torch.randn((rows, 1), device=dev(), dtype=torch.bfloat16)
    q = lib.mxfp4_quantize(x)
    y = lib.mxfp4_dequant(q)
    for first in (0, (1 << 24) - 50, (1 << 25) - 50, (1 << 29) - 100, rows - 100):
        sl = slice(first, first + 100)
        want_c, want_s = MX.quantize(host(x[sl]))
        np.testing.assert_array_equal(q.codes[sl].cpu().numpy(), want_c)
        np.testing.assert_array_equal(q.scales[:, sl].cpu().numpy(), want_s)
        np.testing.assert_array_equal(host(y[sl]), MX.values(host(x[sl])).astype(np.float32))
    del x, q, y
    torch.cuda.empty_cache()


def test_dequant_of_every_code_and_scale():
    """All 16 codes under all 256 scale bytes, to fp32 and bf16 (rounded as the value is: only bytes 253, 254 overflow)."""
    say("mxfp4 dequant of every byte")
    codes = np.zeros((256, 128), dtype=np.uint8)
    codes[:, :16] = np.tile(np.arange(8) * 2 | ((np.arange(8) * 2 + 1) << 4), 2)
    scales = np.zeros((1, 256, 8), dtype=np.uint8)
    scales[0, :, 0] = np.arange(256)
    m = lib.MXMatrix(to_dev(codes), to_dev(scales), 256, 32)
    want = MX.dequant(codes, scales, 32)
    with np.errstate(over="ignore"):
        for kind in ("f32", "bf16"):
            got = host(lib.mxfp4_dequant(m, kind))
            np.testing.assert_array_equal(got[:253].astype(np.float64), want[:253])
            np.testing.assert_array_equal(got[253:255], want[253:255].astype(np.float32))
            assert np.isnan(got[255]).all()


def _inputs(M, N, K, r, seed):
    W = synth.gaussian((N, K), 0.02, synth.SEED_W + seed)
    X = synth.to_bf16(synth.gaussian((M, K), 1.0, synth.SEED_X + seed))
    A = synth.to_bf16(synth.gaussian((max(r, 1), K), 0.05, synth.SEED_A + seed))
    B = synth.to_bf16(synth.gaussian((N, max(r, 1)), 0.05, synth.SEED_B + seed))
    G = synth.to_bf16(synth.gaussian((M, N), 1.0, synth.SEED_DY + seed))
    return W, X, A, B, G


def _ws(op, M, N, K, r):
    n = lib.mx_workspace_size(op, M, N, K, r)
    assert n % 256 == 0
    full, view = guarded(n, torch.uint8)
    view.fill_(0xFF)   # NaN bytes: a value read before it is written shows
    return n, full, view


def run_mx(M, N, K, r, p, give_H=True, backward=True, seed=0):
    """One forward and backward with every output and workspace in guard bands, checked against the oracle."""
    alpha = 2.0 * r
    W, X, A, B, G = _inputs(M, N, K, r, seed)
    w = lib.mxfp4_quantize(to_dev(W))
    d = lib.Dropout(p, SEED, OFF + seed) if p is not None else None
    Xd, Gd = X.to(dev()), G.to(dev())
    Ad, Bd = (A.to(dev()), B.to(dev())) if r else (None, None)
    out = {}
    for name, shape, dt in (("Y", (M, N), torch.bfloat16), ("H", (M, r), torch.float32), ("dX", (M, K), torch.bfloat16),
                            ("dA", (r, K), torch.bfloat16), ("dB", (N, r), torch.bfloat16)):
        nb = int(np.prod(shape)) * (4 if dt == torch.float32 else 2)
        full, view = guarded(nb, dt)
        out[name] = (full, nb, view.view(shape))
    nf, wf, wsf = _ws(lib.QN_OP_FWD, M, N, K, r)
    H = out["H"][2] if r else None
    lib.qlora_mx_linear_fwd(Xd, w, Ad, Bd, alpha, drop=d, Y=out["Y"][2], H=H, ws=wsf)
    assert guards_intact(wf, nf), "forward workspace"
    grads = None
    if backward:
        nbk, wb, wsb = _ws(lib.QN_OP_BWD, M, N, K, r)
        grads = (out["dX"][2],) + ((out["dA"][2], out["dB"][2]) if r else (None, None))
        lib.qlora_mx_linear_bwd(Gd, Xd, w, Ad, Bd, alpha, drop=d, out=grads, ws=wsb, H=H if give_H else None)
        assert guards_intact(wb, nbk), "backward workspace"
    for name, (full, nb, _) in out.items():
        assert guards_intact(full, nb), name
    Xv, Av, Bv, Gv = (synth.bf16_values(t).astype(np.float64) for t in (X, A, B, G))
    What, base = MX.values(W), MX.values(Xv)
    if r == 0:
        Av, Bv, alpha, r = np.zeros((1, K)), np.zeros((N, 1)), 1.0, 1
        keep = None
        zero = torch.zeros
        if grads is not None:
            grads = (grads[0], zero((1, K)), zero((N, 1)))
    else:
        keep = D.keep(M * K, p, SEED, OFF + seed).reshape(M, K) if p is not None else None
    check_step(out["Y"][2], H, grads, Gv, Xv, base, What, Av, Bv, alpha, keep, D.scale(p or 0.0),
               host(H).astype(np.float64) if (H is not None and give_H) else None)
    return out


@pytest.mark.parametrize("M", [1, 2, 3, 8, 15, 16, 17, 31, 32])
@pytest.mark.parametrize("N, K, r, p", [(64, 64, 8, None), (192, 320, 13, 0.25), (128, 1088, 64, None), (64, 2112, 0, None),
                                        (320, 4160, 16, 0.1)])
def test_few_rows(M, N, K, r, p):
    say(f"mx linear M={M} N={N} K={K} r={r} p={p}")
    run_mx(M, N, K, r, p, seed=M)


@pytest.mark.parametrize("M, N, K, r, p", [(1, 128, 8256, 8, None), (7, 64, 16448, 0, None), (16, 8192, 1024, 16, None),
                                           (2, 16384, 256, 0, None), (5, 12352, 192, 24, 0.5),
                                           (20, 128, 8256, 13, 0.25), (32, 16384, 256, 64, None),
                                           (25, 33024, 64, 8, 0.1)])
def test_few_rows_long_rows_and_many_rows_of_weight(M, N, K, r, p):
    """Split columns (K beyond 8192) and two and four row groups per wave."""
    say(f"mx linear M={M} N={N} K={K} r={r} p={p}")
    run_mx(M, N, K, r, p, backward=False, seed=M)


@pytest.mark.parametrize("M", [33, 64, 127, 128, 129, 300])
@pytest.mark.parametrize("N, K, r, p, give_H", [(64, 64, 8, None, True), (192, 320, 13, 0.25, False),
                                                (448, 1088, 64, 0.5, True), (128, 704, 0, None, True),
                                                (64, 192, 33, None, False)])
def test_tiles(M, N, K, r, p, give_H):
    say(f"mx linear M={M} N={N} K={K} r={r} p={p} give_H={give_H}")
    run_mx(M, N, K, r, p, give_H=give_H, seed=M)


@pytest.mark.parametrize("M, N, K, r, p", [(17, 64, 4096, 16, 0.1), (40, 4096, 64, 20, None), (200, 256, 2304, 0, None),
                                           (33, 64, 4096, 16, 0.1), (100, 192, 2304, 13, 0.25), (128, 64, 1600, 64, None),
                                           (200, 64, 4096, 24, 0.1), (1000, 128, 2112, 5, 0.5)])
def test_split_contractions(M, N, K, r, p):
    """Long contractions of small outputs, forward (over K) and dX (over N)."""
    say(f"mx linear split M={M} N={N} K={K} r={r} p={p}")
    run_mx(M, N, K, r, p, seed=M)


@pytest.mark.parametrize("r, p", [(16, 0.2), (64, None), (5, 0.5), (0, None)])
def test_large_tiles(r, p):
    """Shapes that take the 256 x 256 tiles, with ragged edges on every side, forward and dX."""
    say(f"mx linear large tiles r={r} p={p}")
    run_mx(2200, 4160, 320, r, p, seed=r)
    run_mx(2100, 320, 4160, r, p, seed=r + 1)


@pytest.mark.parametrize("M, N, K, r, p", [(100, 512, 320, 16, 0.3), (801, 512, 704, 9, None), (2700, 3584, 320, 40, 0.1),
                                           (2650, 3584, 320, 5, None), (3290, 512, 1088, 16, 0.5), (3300, 3584, 1088, 8, 0.2),
                                           (3270, 3584, 1088, 0, None), (3570, 512, 2304, 24, None)])
def test_dX_tile_heights_and_cuts(M, N, K, r, p):
    """dX on tiles of 64, 128 and 256 rows, cut over N or not, with and without a mask."""
    say(f"mx dX plans M={M} N={N} K={K} r={r} p={p}")
    run_mx(M, N, K, r, p, seed=r)


@pytest.mark.parametrize("r, p", [(16, 0.2), (0, None)])
def test_large_and_small_tiles_in_one_call(r, p):
    """A last round that is mostly empty: whole columns of it go to the small tiles, a second launch at column offsets."""
    say(f"mx linear mixed tiles r={r} p={p}")
    run_mx(2200, 8448, 704, r, p, backward=False, seed=r)


@pytest.mark.parametrize("M", [4, 40, 300])
def test_non_finite_rows_stay_in_their_row(M):
    say(f"mx linear with a non-finite row, M={M}")
    N, K = 128, 320
    W, X, _, _, _ = _inputs(M, N, K, 0, 1)
    w = lib.mxfp4_quantize(to_dev(W))
    clean = lib.qlora_mx_linear_fwd(X.to(dev()), w)
    X[2, 100] = float("nan")
    X[3, 319] = float("inf")
    Y = lib.qlora_mx_linear_fwd(X.to(dev()), w)
    torch.cuda.synchronize()
    rows = torch.ones(M, dtype=torch.bool)
    rows[2] = rows[3] = False
    assert torch.isnan(Y[2:4]).all() and torch.equal(Y.cpu()[rows], clean.cpu()[rows])


@pytest.mark.parametrize("M", [9, 200])
def test_masked_infinities_reach_no_adapter_gradient(M):
    say(f"mx linear, infinities at dropped positions, M={M}")
    N, K, r, p = 64, 128, 8, 0.4
    W, X, A, B, G = _inputs(M, N, K, r, 3)
    keep = torch.from_numpy(D.keep(M * K, p, SEED, OFF).reshape(M, K))
    w, d = lib.mxfp4_quantize(to_dev(W)), lib.Dropout(p, SEED, OFF)
    A, B, G = A.to(dev()), B.to(dev()), G.to(dev())
    res = []
    for fill in (float("nan"), 0.0):
        Xf = torch.where(keep, X, torch.full_like(X, fill)).to(dev())
        _, H = lib.qlora_mx_linear_fwd(Xf, w, A, B, 16.0, drop=d, want_H=True)
        res.append((H,) + lib.qlora_mx_linear_bwd(G, Xf, w, A, B, 16.0, drop=d))
    for a, b in zip(*res):
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("M", [3, 90])
def test_repeats_streams_and_concurrent_calls(M):
    """Bit-equal repeats, also with two calls on two other streams at once (a workspace each)."""
    say(f"mx linear streams M={M}")
    N, K, r = 256, 1088, 16
    W, X, A, B, G = _inputs(M, N, K, r, 4)
    w = lib.mxfp4_quantize(to_dev(W))
    X, A, B, G = (t.to(dev()) for t in (X, A, B, G))
    d = lib.Dropout(0.2, SEED, OFF)
    Y, H = lib.qlora_mx_linear_fwd(X, w, A, B, 32.0, drop=d, want_H=True)
    ref = (Y, H) + lib.qlora_mx_linear_bwd(G, X, w, A, B, 32.0, drop=d, H=H)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for s in streams:
        with torch.cuda.stream(s):
            Y, H = lib.qlora_mx_linear_fwd(X, w, A, B, 32.0, drop=d, want_H=True)
            outs.append((Y, H) + lib.qlora_mx_linear_bwd(G, X, w, A, B, 32.0, drop=d, H=H))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, ref))


@pytest.mark.parametrize("M", [4, 200])
def test_training_step_captured_and_replayed(M):
    """Quantise, forward, backward and the optimizer step in one graph, a mask per
    replay through offset_dev, against the same calls made eagerly."""
    say(f"mx training step under capture M={M}")
    N, K, r, alpha = 192, 576, 16, 32.0
    W, X, A, B, G = (t if isinstance(t, np.ndarray) else t.to(dev()) for t in _inputs(M, N, K, r, 6))
    W = to_dev(W)

    def setup():
        st = dict(A=A.clone(), B=B.clone(), w=lib.MXMatrix.empty(N, K, dev()),
                  step=torch.zeros(1, dtype=torch.int64, device=dev()),
                  Y=torch.empty((M, N), dtype=torch.bfloat16, device=dev()), H=torch.empty((M, r), device=dev()),
                  g=tuple(torch.empty(s, dtype=torch.bfloat16, device=dev()) for s in ((M, K), (r, K), (N, r))),
                  wf=lib.mx_workspace(lib.QN_OP_FWD, M, N, K, r, dev()),
                  wb=lib.mx_workspace(lib.QN_OP_BWD, M, N, K, r, dev()),
                  oA=lib.AdamW8State(A.numel(), dev()), oB=lib.AdamW8State(B.numel(), dev()))
        st["d"] = lib.Dropout(0.3, SEED, OFF, offset_dev=st["step"])
        return st

    def body(st):
        lib.mxfp4_quantize(W, out=st["w"])
        lib.qlora_mx_linear_fwd(X, st["w"], st["A"], st["B"], alpha, drop=st["d"], Y=st["Y"], H=st["H"], ws=st["wf"])
        lib.qlora_mx_linear_bwd(G, X, st["w"], st["A"], st["B"], alpha, drop=st["d"], out=st["g"], ws=st["wb"], H=st["H"])
        lib.adamw8_step_multi([st["A"], st["B"]], [st["g"][1], st["g"][2]], [st["oA"], st["oB"]], lr=1e-3, step=2)
        st["step"].add_(1)

    cap, eager = setup(), setup()
    body(cap)
    body(eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        body(cap)
    last = None
    for rep in range(3):
        graph.replay()
        body(eager)
        other = torch.ones(4096, device=dev()).sum()
        torch.cuda.synchronize()
        assert float(other) == 4096.0
        for k in ("Y", "H", "A", "B", "step"):
            assert torch.equal(cap[k], eager[k]), f"replay {rep}: {k}"
        assert all(torch.equal(a, b) for a, b in zip(cap["g"], eager["g"])), f"replay {rep}: gradients"
        assert last is None or not torch.equal(cap["H"], last)
        last = cap["H"].clone()


def test_adapter_gradient_against_differences():
    """dB and dA of a sum of G * Y, by moving one adapter element up and down: the
    forward is linear in it, so the difference is exact but for Y's bf16 rounding,
    2^-8 |Y| per element and side, weighted by |G| and divided by the distance."""
    say("mx linear adapter gradients against differences")
    M, N, K, r = 24, 64, 128, 8
    W, X, A, B, G = _inputs(M, N, K, r, 8)
    w = lib.mxfp4_quantize(to_dev(W))
    d = lib.Dropout(0.25, SEED, OFF)
    Xd, Gd = X.to(dev()), G.to(dev())
    _, dA, dB = lib.qlora_mx_linear_bwd(Gd, Xd, w, A.to(dev()), B.to(dev()), 16.0, drop=d)
    for t, g, at in ((A, dA, (3, 17)), (A, dA, (7, 120)), (B, dB, (5, 2)), (B, dB, (63, 7))):
        vals, noise, x = [], 0.0, []
        for h in (8.0, -8.0):
            u = t.clone()
            u[at] = h
            x.append(float(u[at]))
            a, b = (u, B) if t is A else (A, u)
            Y = host(lib.qlora_mx_linear_fwd(Xd, w, a.to(dev()), b.to(dev()), 16.0, drop=d)).astype(np.float64)
            Gv = synth.bf16_values(G).astype(np.float64)
            vals.append((Y * Gv).sum())
            # Y's rounding, and that of bf16(s H) under B (the moved element dominates both)
            noise += (2.0 ** -8 * np.abs(Y) * np.abs(Gv)).sum() * 2
        got, ref = float(g[at]), (vals[0] - vals[1]) / (x[0] - x[1])
        assert abs(got - ref) <= noise / (x[0] - x[1]) + 2.0 ** -7 * abs(ref) + 1e-3


def test_python_refusals_on_the_device():
    say("mx linear refusals")
    X = torch.zeros((4, 128), dtype=torch.bfloat16, device=dev())
    w = lib.mxfp4_quantize(torch.zeros((64, 128), device=dev()))
    A = torch.zeros((8, 128), dtype=torch.bfloat16, device=dev())
    B = torch.zeros((64, 8), dtype=torch.bfloat16, device=dev())
    with pytest.raises(ValueError):
        lib.qlora_mx_linear_fwd(X, w, A, None, 1.0)
    with pytest.raises(ValueError):
        lib.qlora_mx_linear_fwd(X[:, :64].contiguous(), w, A, B, 1.0)
    with pytest.raises(ValueError):
        lib.qlora_mx_linear_fwd(X[:, ::2], w, A, B, 1.0)
    with pytest.raises(ValueError):
        lib.qlora_mx_linear_fwd(X, w, A, B, 1.0, Y=torch.empty((4, 32), dtype=torch.bfloat16, device=dev()))
    with pytest.raises(ValueError):
        lib.qlora_mx_linear_fwd(X, w, want_H=True)
    with pytest.raises(lib.QNError):
        lib.qlora_mx_linear_fwd(X, w, A, B, 1.0, ws=torch.empty(16, dtype=torch.uint8, device=dev()))
    with pytest.raises(lib.QNError):
        lib.dropout(X, lib.Dropout(1.0, 0))
    with pytest.raises(ValueError):
        lib.qlora_mx_linear_fwd(X, w, A.cpu(), B, 1.0)
    with pytest.raises(ValueError):
        lib.qlora_mx_linear_bwd(torch.zeros((4, 64), dtype=torch.bfloat16, device=dev()), X, w, A, B, 1.0,
                                out=(None, None, None))


def test_rows_beyond_32_bits():
    """X and dX of more than 2^32 bytes: sampled rows of Y, H and dX, all of dA and dB."""
    M, N, K, r = (1 << 20) + 77, 64, 2048, 8
    say(f"mx linear M={M} N={N} K={K}")
    W, _, A, B, _ = _inputs(1, N, K, r, 2)
    w = lib.mxfp4_quantize(to_dev(W))
    gen = torch.Generator(device=dev()).manual_seed(7)
    X = torch.randn((M, K), generator=gen, device=dev(), dtype=torch.bfloat16)
    G = torch.randn((M, N), generator=gen, device=dev(), dtype=torch.bfloat16)
    A, B, alpha = A.to(dev()), B.to(dev()), 16.0
    Y, H = lib.qlora_mx_linear_fwd(X, w, A, B, alpha, want_H=True)
    dX, dA, dB = lib.qlora_mx_linear_bwd(G, X, w, A, B, alpha, H=H)
    torch.cuda.synchronize()
    rows = torch.tensor([0, 1, 255, 256, (1 << 19) - 1, 1 << 19, (1 << 20) - 1, 1 << 20, M - 78, M - 2, M - 1], device=dev())
    Xv, Gv, Av, Bv = (host(t).astype(np.float64) for t in (X[rows], G[rows], A, B))
    Hv, What = host(H[rows]).astype(np.float64), MX.values(W)
    check_step(Y[rows], H[rows], None, Gv, Xv, MX.values(Xv), What, Av, Bv, alpha, None, 1.0, Hv)
    s, ab = alpha / r, np.abs
    dH = s * (Gv @ Bv)
    # dX: its own rounding, fp32 sums of N and r terms, dH rounded to bf16
    tol = HALF * ab(Gv @ What + dH @ Av) + N * EPS * (ab(Gv) @ ab(What)) + (HALF + (N + r) * EPS) * ((s * (ab(Gv) @ ab(Bv))) @ ab(Av))
    assert np.all(ab(host(dX[rows]).astype(np.float64) - (Gv @ What + dH @ Av)) <= tol)
    # dA = dH^T X and dB = s G^T H in 64 bits, a slab of rows at a time
    rA, rB = (torch.zeros(t, dtype=torch.float64, device=dev()) for t in ((r, K), (N, r)))
    for m in range(0, M, 1 << 17):
        x, g, h = (t[m:m + (1 << 17)].double() for t in (X, G, H))
        rA += (s * (g @ B.double())).t() @ x
        rB += s * (g.t() @ h)
    assert rel_fro(host(dA), rA.cpu().numpy()) <= REL_FRO_TOL
    assert rel_fro(host(dB), rB.cpu().numpy()) <= REL_FRO_TOL
