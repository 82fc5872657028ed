"""GPU parity of the norm of queries and keys per head with the position rotation, and its gradients, with the float64
oracle, elementwise against bounds derived from the evaluation's roundings (oracle.norm_rope.error_bounds)."""

import numpy as np
import pytest

import tiled_genome_diffusion_amd as pc
from gpu_util import say, torch_dev
from oracle import norm_rope as nr

pytestmark = pytest.mark.gpu

# relative rounding of the type, and the absolute one below its normal range
UNIT = {"float32": (2.0 ** -24, 0.0), "bfloat16": (2.0 ** -8, 0.0), "float16": (2.0 ** -11, 2.0 ** -25)}


def freqs_of(n):
    return 10000.0 ** (-np.arange(n) / max(n, 1))


def make(dtype, B, L, H, D, seed, positions="batch", weight=True):
    torch, dev = torch_dev()
    gen = torch.Generator().manual_seed(seed)
    s = {"x": torch.randn(B, L, H, D, generator=gen).to(getattr(torch, dtype)).to(dev),
         "dy": torch.randn(B, L, H, D, generator=gen).to(getattr(torch, dtype)).to(dev),
         "w": (1.0 + 0.2 * torch.randn(D, generator=gen)).to(dev) if weight else None, "pos": None}
    if positions == "batch":
        s["pos"] = torch.randint(-5000, 5000, (B, L), generator=gen, dtype=torch.int32).to(dev)
    elif positions == "shared":
        s["pos"] = torch.randint(0, 2000, (L,), generator=gen, dtype=torch.int32).to(dev)
    return s


def f64(t):
    return t.double().cpu().numpy()


def reference(s):
    B, L, _, D = s["x"].shape
    w = np.ones(D) if s["w"] is None else f64(s["w"])
    pos = np.broadcast_to(np.arange(L) if s["pos"] is None else s["pos"].cpu().numpy(), (B, L))
    return f64(s["x"]), w, pos, f64(s["dy"])


def check(name, got, want, bound):
    err = np.abs(f64(got) - want)
    assert np.isfinite(f64(got)).all(), f"{name} holds values that are not finite"
    over = (err - bound).max(initial=-np.inf)
    assert over <= 0.0, f"{name}: over its bound by {over:.3e} (largest error {err.max():.3e})"


def run_both(q, k, freqs, eps, inter):
    """Outputs, input gradients and weight gradients of both sides (None where a side is absent)."""
    torch, dev = torch_dev()
    like = lambda s: None if s is None else torch.full(s["x"].shape, 7.0, dtype=s["x"].dtype, device=dev)  # noqa: E731
    get = lambda s, n: None if s is None else s[n]  # noqa: E731
    y, dx = [like(q), like(k)], [like(q), like(k)]
    dw = [None if s is None else torch.full((s["x"].shape[3],), 7.0, device=dev) for s in (q, k)]
    sides = (get(q, "x"), get(k, "x"), get(q, "w"), get(k, "w"), get(q, "pos"), get(k, "pos"), freqs)
    pc.pc_qk_norm_rope(*sides, *y, eps=eps, interleaved=inter)
    pc.pc_qk_norm_rope_backward(*sides, get(q, "dy"), get(k, "dy"), *dx, *dw, eps=eps, interleaved=inter)
    return y, dx, dw


def check_case(q, k, n_pairs, eps, inter, dtype):
    f, e = freqs_of(n_pairs), float(np.float32(eps))
    for s, y, dx, dw in zip((q, k), *run_both(q, k, f, eps, inter)):
        if s is None:
            continue
        x, w, pos, dy = reference(s)
        b = nr.error_bounds(x, w, pos, f, e, inter, dy, *UNIT[dtype])
        check("y", y, nr.forward(x, w, pos, f, e, inter), b[0])
        want = nr.backward(x, w, pos, f, e, inter, dy)
        check("dx", dx, want[0], b[1])
        check("dweight", dw, want[1], b[2])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("dim,rot", [(8, 0), (16, 16), (32, 32), (40, 32), (64, 64), (64, 16), (72, 48), (96, 96),
                                     (128, 64), (128, 128)])
def test_head_sizes(dim, rot, dtype, inter):
    say(f"norm + rotation, {dtype}, heads of {dim}, {rot} rotated, interleaved {inter}")
    check_case(make(dtype, 3, 7, 4, dim, dim), make(dtype, 2, 33, 2, dim, dim + 1, "shared"), rot // 2, 1e-6, inter, dtype)


@pytest.mark.parametrize("B,L,H", [(1, 1, 1), (1, 1, 16), (5, 1, 3), (1, 300, 1), (2, 64, 8), (9, 65, 5), (70, 64, 12)])
def test_shapes(B, L, H):
    say(f"norm + rotation, [{B}][{L}][{H}]")
    for dtype in ("float32", "bfloat16"):
        check_case(make(dtype, B, L, H, 64, B), None, 32, 1e-6, False, dtype)
        check_case(None, make(dtype, B, L, H, 64, B, "none", weight=False), 16, 1e-2, True, dtype)


def test_more_tiles_than_workgroups():
    """The gradients' workgroups take several tiles each."""
    torch, dev = torch_dev()
    say("norm + rotation, 40,000 tokens of 16 heads")
    q = make("bfloat16", 40, 1000, 16, 128, 3)
    check_case(q, make("bfloat16", 1, 5, 16, 128, 4), 64, 1e-6, False, "bfloat16")


def test_positions_of_a_whole_chain():
    """Positions up to the ends of int32: the angle keeps its digits."""
    torch, dev = torch_dev()
    say("norm + rotation, positions near +-2^31")
    q = make("float32", 1, 6, 2, 64, 5)
    q["pos"] = torch.tensor([[2 ** 31 - 1, -2 ** 31, 10 ** 9, 123456789, -1, 0]], dtype=torch.int32, device=dev)
    # the oracle's own float64 angle is good to 2^31 2^-53 radians
    check_case(q, None, 32, 1e-6, False, "float32")


def test_zero_rows_and_infinities():
    torch, dev = torch_dev()
    say("norm + rotation, rows of zeros, NaN")
    q = make("float32", 1, 4, 2, 32, 6)
    q["x"][0, 1] = 0.0
    check_case(q, None, 16, 1e-6, False, "float32")
    clean = run_both(q, None, freqs_of(16), 1e-6, False)[0][0].clone()
    q["x"][0, 2, 1, 5] = float("nan")
    y = run_both(q, None, freqs_of(16), 1e-6, False)[0][0]
    assert torch.isnan(y[0, 2, 1]).all()
    y[0, 2, 1] = clean[0, 2, 1]
    assert torch.equal(y, clean)


def test_strided_in_place_and_empty():
    torch, dev = torch_dev()
    say("norm + rotation, strided, in place, empty")
    for dtype in ("float32", "bfloat16"):
        q, k = make(dtype, 3, 20, 4, 72, 7), make(dtype, 3, 31, 4, 72, 8)
        f = freqs_of(32)
        (yq, yk), (dq, dk), (dwq, dwk) = run_both(q, k, f, 1e-6, False)
        both = torch.cat([q["x"], make(dtype, 3, 20, 4, 72, 9)["x"]], dim=2)      # queries beside other heads
        view = both[:, :, :4]
        rest = both[:, :, 4:].clone()
        kt = k["x"].transpose(1, 2).contiguous().transpose(1, 2)
        pc.pc_qk_norm_rope(view, kt, q["w"], k["w"], q["pos"], k["pos"], f, view, kt)   # in place
        assert torch.equal(view, yq) and torch.equal(kt, yk) and torch.equal(both[:, :, 4:], rest)
        gq = q["dy"].clone()
        dw = torch.empty_like(dwq)
        pc.pc_qk_norm_rope_backward(q["x"], None, q["w"], None, q["pos"], None, f, gq, None, gq, None, dw)
        assert torch.equal(gq, dq) and torch.equal(dw, dwq)
        ones = torch.ones(1, 1, 1, 72, dtype=q["x"].dtype, device=dev)
        g = torch.empty_like(dq)
        pc.pc_qk_norm_rope_backward(q["x"], None, q["w"], None, q["pos"], None, f, ones.expand(3, 20, 4, 72), None, g, None)
        h = torch.empty_like(dq)
        pc.pc_qk_norm_rope_backward(q["x"], None, q["w"], None, q["pos"], None, f, torch.ones_like(dq), None, h, None)
        assert torch.equal(g, h)                                                   # a broadcast gradient
    e = torch.empty(0, 5, 2, 32, device=dev)
    dw = torch.full((32,), 7.0, device=dev)
    pc.pc_qk_norm_rope(e, None, None, None, None, None, freqs_of(8), e, None)
    pc.pc_qk_norm_rope_backward(e, None, None, None, None, None, freqs_of(8), e, None, e, None, dw)
    assert not dw.any()


def test_runs_are_identical_in_slices_streams_and_graphs():
    torch, dev = torch_dev()
    say("norm + rotation, repeated / sliced / side stream / graph")
    q, k = make("bfloat16", 30, 64, 8, 64, 10), make("bfloat16", 3, 200, 4, 64, 11)
    f = freqs_of(32)
    want = [t for part in run_both(q, k, f, 1e-6, False) for t in part]

    def same(got):
        return all(torch.equal(a, b) for a, b in zip(want, [t for part in got for t in part]))

    assert same(run_both(q, k, f, 1e-6, False))
    pc.pc_set_max_dispatch_items(1024)
    try:
        assert same(run_both(q, k, f, 1e-6, False))
    finally:
        pc.pc_set_max_dispatch_items(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run_both(q, k, f, 1e-6, False)
    torch.cuda.current_stream().wait_stream(side)
    assert same(got)
    bufs = [torch.empty_like(t) for t in want]
    ws = torch.empty(pc.pc_qk_norm_rope_workspace(q["x"], k["x"], f), dtype=torch.uint8, device=dev)
    sides = (q["x"], k["x"], q["w"], k["w"], q["pos"], k["pos"], f)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pc.pc_qk_norm_rope(*sides, bufs[0], bufs[1])
        pc.pc_qk_norm_rope_backward(*sides, q["dy"], k["dy"], *bufs[2:], workspace=ws)
    for n in range(3):
        for t in bufs:
            t.fill_(float(n))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, bufs)), f"replay {n}"


def test_binding_refuses():
    torch, dev = torch_dev()
    say("norm + rotation, refusals of the binding")
    q, k = make("bfloat16", 2, 5, 2, 64, 12), make("bfloat16", 2, 5, 2, 32, 13)
    f = freqs_of(32)
    x, w = q["x"], q["w"]
    y = torch.empty_like(x)
    for g in (lambda: pc.pc_qk_norm_rope(None, None, None, None, None, None, f, None, None),
              lambda: pc.pc_qk_norm_rope(x, k["x"], w, k["w"], None, None, f, y, k["x"]),
              lambda: pc.pc_qk_norm_rope(x, None, w.bfloat16(), None, None, None, f, y, None),
              lambda: pc.pc_qk_norm_rope(x, None, w, None, torch.zeros(3, 5, dtype=torch.int32, device=dev), None, f, y, None),
              lambda: pc.pc_qk_norm_rope(x, None, w, None, torch.zeros(5, device=dev), None, f, y, None),
              lambda: pc.pc_qk_norm_rope(x, None, w, None, None, None, f, y.float(), None)):
        with pytest.raises(ValueError):
            g()
    for g in (lambda: pc.pc_qk_norm_rope(x, None, w, None, None, None, freqs_of(12), y, None),
              lambda: pc.pc_qk_norm_rope(x, None, w, None, None, None, freqs_of(40), y, None),
              lambda: pc.pc_qk_norm_rope(x, None, w, None, None, None, np.full(32, 7.0), y, None),
              lambda: pc.pc_qk_norm_rope(x, None, w, None, None, None, np.full(32, np.nan), y, None),
              lambda: pc.pc_qk_norm_rope(x, None, w, None, None, None, f, y, None, eps=-1.0),
              lambda: pc.pc_qk_norm_rope_backward(x, None, w, None, None, None, f, y, None, x.clone(), None,
                                                  torch.empty(64, device=dev), workspace=torch.empty(16, dtype=torch.uint8,
                                                                                                     device=dev))):
        with pytest.raises(pc.PCError):
            g()
