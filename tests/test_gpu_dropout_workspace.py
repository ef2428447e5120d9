"""GPU: the backward with dropout in a workspace of its own op (dX's contraction cut
where few tiles would leave compute units idle) and in the plain backward's (never
cut), and the plain backward in exactly its own, all poisoned and in guard bands.
Tolerances as test_gpu_dropout.py derives them."""

import numpy as np
import pytest
import torch

import oracle
from bit_nf4_quantized_08_amd import lib, synth
from oracle import dropout as D
from tests.gpu_util import dev, guarded, guards_intact, host, say, to_dev
from tests.test_gpu_dropout import OFF, SEED, check_step

pytestmark = pytest.mark.gpu


def _inputs(M, N, K, r, seed):
    W = synth.gaussian((N, K), 0.02, synth.SEED_W + seed)
    X = synth.to_bf16(synth.gaussian((M, K), 1.0, synth.SEED_X + seed))
    A = synth.to_bf16(synth.gaussian((r, K), 0.05, synth.SEED_A + seed))
    B = synth.to_bf16(synth.gaussian((N, r), 0.05, synth.SEED_B + seed))
    G = synth.to_bf16(synth.gaussian((M, N), 1.0, synth.SEED_DY + seed))
    return W, X, A, B, G


# room: only the larger workspace has room for dX's partial products
@pytest.mark.parametrize("M, N, K, r, p, room", [
    (61, 1088, 1344, 24, 0.25, True), (260, 1216, 1152, 40, 0.1, True), (300, 4160, 576, 64, 0.05, True),
    (70, 1088, 1088, 16, 0.0, True), (1, 1024, 1024, 1, 0.1, False), (5, 704, 2112, 8, 0.5, False),
    (8, 64, 64, 32, 0.2, False), (1, 64, 64, 64, 0.2, False), (129, 64, 192, 33, 0.4, False),
])
@pytest.mark.parametrize("give_H", [True, False])
def test_both_sizes(M, N, K, r, p, room, give_H):
    say(f"nf4 dropout backward, both workspaces, M={M} N={N} K={K} r={r} p={p} give_H={give_H}")
    alpha = 2.0 * r
    W, X, A, B, G = _inputs(M, N, K, r, M + r)
    w, d = lib.quantize_weight(to_dev(W)), lib.Dropout(p, SEED, OFF)
    Xd, Ad, Bd, Gd = (t.to(dev()) for t in (X, A, B, G))
    Xv, Av, Bv, Gv = (synth.bf16_values(t).astype(np.float64) for t in (X, A, B, G))
    p_, a_, _ = oracle.quantize(W)
    What = oracle.dequant_bf16_weight(p_, N, K, oracle.dq_absmax(*oracle.double_quant(a_))).astype(np.float64)
    keep = D.keep(M * K, p, SEED, OFF).reshape(M, K)
    H = (D.scale(p) * np.where(keep, Xv, 0.0) @ Av.T).astype(np.float32)
    small, large = (lib.workspace_size(op, M, N, K, r) for op in (lib.QN_OP_BWD, lib.QN_OP_BWD_DROPOUT))
    assert (large > small) == room
    dX = []
    for n in (small, large):
        full, ws = guarded(n, torch.uint8)
        ws.fill_(0xFF)
        grads = lib.qlora_linear_bwd_dropout(Gd, Xd, w, Ad, Bd, alpha, d, ws=ws, H=to_dev(H) if give_H else None)
        assert guards_intact(full, n)
        check_step(None, None, grads, Gv, Xv, Xv, What, Av, Bv, alpha, keep, D.scale(p),
                   H.astype(np.float64) if give_H else None)
        dX.append(grads[0])
    if not room:   # the same plan in both
        assert torch.equal(*dX)


@pytest.mark.parametrize("M, N, K, r", [(512, 1088, 1344, 24), (5, 704, 2112, 8), (300, 512, 320, 64)])
def test_plain_backward_in_its_own_size(M, N, K, r):
    """The plain backward in exactly the bytes it asks for: results as in a roomy workspace, nothing written outside."""
    say(f"plain backward workspace M={M} N={N} K={K} r={r}")
    W, X, A, B, G = (t if isinstance(t, np.ndarray) else t.to(dev()) for t in _inputs(M, N, K, r, 2))
    w = lib.quantize_weight(to_dev(W))
    n = lib.workspace_size(lib.QN_OP_BWD, M, N, K, r)
    full, ws = guarded(n, torch.uint8)
    ws.fill_(0xFF)
    got = lib.qlora_linear_bwd(G, X, w, A, B, 16.0, ws=ws)
    assert guards_intact(full, n)
    ref = lib.qlora_linear_bwd(G, X, w, A, B, 16.0, ws=torch.empty(2 * n, dtype=torch.uint8, device=dev()))
    for a, b in zip(got, ref):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_cut_backward_captured_and_replayed():
    """The cut contraction in a graph, a mask per replay, against the same calls made eagerly."""
    M, N, K, r = 61, 1088, 1344, 24
    say("nf4 dropout, cut dX under capture")
    W, X, A, B, G = (t if isinstance(t, np.ndarray) else t.to(dev()) for t in _inputs(M, N, K, r, 4))
    w = lib.quantize_weight(to_dev(W))

    def setup():
        step = torch.zeros(1, dtype=torch.int64, device=dev())
        return dict(step=step, d=lib.Dropout(0.2, SEED, OFF, offset_dev=step),
                    g=tuple(torch.zeros(t, dtype=torch.bfloat16, device=dev()) for t in ((M, K), (r, K), (N, r))),
                    ws=lib.workspace(lib.QN_OP_BWD_DROPOUT, M, N, K, r, dev()))

    def body(st):
        lib.qlora_linear_bwd_dropout(G, X, w, A, B, 16.0, st["d"], out=st["g"], ws=st["ws"])
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
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(cap["g"] + (cap["step"],), eager["g"] + (eager["step"],))), rep
        assert last is None or not torch.equal(cap["g"][1], last)
        last = cap["g"][1].clone()
