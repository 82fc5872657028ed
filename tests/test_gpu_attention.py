"""GPU parity of cross attention and its gradients with the float64 oracle.

Every comparison is elementwise against a bound derived from the evaluation's roundings (oracle.attention.error_bounds):
float32 scores, statistics and sums, P and dS rounded to the tensors' type for their products, results rounded once.
"""

import numpy as np
import pytest

import tiled_genome_diffusion_amd as pc
from gpu_util import say, torch_dev
from oracle import attention as att

pytestmark = pytest.mark.gpu

# relative rounding of results and of P and dS, and the absolute one below the type's normal range (2^-126 in 32 bits,
# where the hardware's exp2 gives 0)
UNIT = {"float32": (2.0 ** -24, 0.0, 2.0 ** -126), "bfloat16": (2.0 ** -8, 2.0 ** -8, 2.0 ** -126),
        "float16": (2.0 ** -11, 2.0 ** -11, 2.0 ** -25)}


def make(dtype, R, G, Lq, Lk, H, Hk, D, mask, seed=0, scale=None, amp=1.0):
    torch, dev = torch_dev()
    dt = getattr(torch, dtype)
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: (amp * torch.randn(*s, generator=gen)).to(dt).to(dev)  # noqa: E731
    c = {"q": n(R * G, Lq, H, D), "k": n(R, Lk, Hk, D), "v": n(R, Lk, Hk, D), "dout": n(R * G, Lq, H, D),
         "kv_len": None, "key_mask": None, "scale": scale or D ** -0.5, "dtype": dtype}
    if mask in ("ragged", "both"):
        c["kv_len"] = torch.randint(0, Lk + 1, (R,), generator=gen, dtype=torch.int32).to(dev)
    if mask in ("holes", "both"):
        c["key_mask"] = (torch.rand(R, Lk, generator=gen) < 0.7).to(torch.uint8).to(dev)
        if R > 1:
            c["key_mask"][1] = 0
    return c


def forward(c, with_lse=True, **kw):
    torch, dev = torch_dev()
    q = c["q"]
    out = torch.full_like(q, 7.0) if q.is_contiguous() else torch.empty_strided(q.shape, q.stride(), dtype=q.dtype,
                                                                              device=dev).fill_(7.0)
    lse = torch.full(q.shape[:3], 7.0, device=dev) if with_lse else None
    pc.pc_cross_attention(q, c["k"], c["v"], out, lse, c["kv_len"], c["key_mask"], c["scale"], **kw)
    return out, lse


def backward(c, out, lse, **kw):
    torch, dev = torch_dev()
    g = [torch.full(c[n].shape, 7.0, dtype=c["q"].dtype, device=dev) for n in "qkv"]
    pc.pc_cross_attention_backward(c["q"], c["k"], c["v"], out, lse, c["dout"], *g, c["kv_len"], c["key_mask"],
                                   c["scale"], **kw)
    return g


def f64(t):
    return t.double().cpu().numpy()


def keep_of(c):
    R, Lk = c["k"].shape[:2]
    cpu = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    return att.attended(R, Lk, cpu(c["kv_len"]), cpu(c["key_mask"]))


def check(name, got, want, bound):
    err = np.abs(f64(got) - want)
    worst = float((err - bound).max(initial=-np.inf))
    assert np.isfinite(f64(got)).all(), f"{name} holds values that are not finite"
    assert worst <= 0.0, f"{name}: error {err.flat[(err - bound).argmax()]:.3e} over its bound by {worst:.3e}"


def check_case(c, train=True):
    u, up, ap = UNIT[c["dtype"]]
    q, k, v, g = (f64(c[n]) for n in ("q", "k", "v", "dout"))
    keep, s = keep_of(c), float(np.float32(c["scale"]))
    want, want_lse = att.forward(q, k, v, keep, s)
    bounds = att.error_bounds(q, k, v, g, keep, s, u, up, ap)
    out, lse = forward(c)
    check("out", out, want, bounds[0])
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(f64(lse)), empty)
    top = np.abs(want_lse[~empty]).max(initial=1.0)
    assert np.abs(f64(lse)[~empty] - want_lse[~empty]).max(initial=0.0) <= 1e-5 * top + 1e-5
    if train:
        for n, got, w, b in zip(("dq", "dk", "dv"), backward(c, out, lse), att.backward(q, k, v, g, keep, s), bounds[1:]):
            check(n, got, w, b)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("dim", [8, 32, 40, 64, 72, 96, 104, 128])
def test_head_sizes(dtype, dim):
    say(f"attention, {dtype}, heads of {dim}")
    check_case(make(dtype, 2, 3, 21, 75, 4, 2, dim, "both", seed=dim))


@pytest.mark.parametrize("mask", ["none", "ragged", "holes", "both"])
@pytest.mark.parametrize("len_k", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300])
def test_key_lengths(len_k, mask):
    say(f"attention, {len_k} keys, mask {mask}")
    for dtype in ("float32", "bfloat16"):
        check_case(make(dtype, 3, 2, 17, len_k, 2, 2, 64, mask, seed=len_k))


@pytest.mark.parametrize("group,len_q,heads,heads_kv", [
    (1, 1, 1, 1), (1, 1, 8, 1), (1, 1, 8, 8), (5, 1, 4, 2), (1, 31, 1, 1), (1, 128, 2, 1), (1, 129, 2, 1),
    (3, 43, 3, 3), (2, 64, 6, 2), (7, 64, 1, 1)])
def test_rows(group, len_q, heads, heads_kv):
    say(f"attention, group {group}, {len_q} tokens, heads {heads}/{heads_kv}")
    for dtype in ("float32", "bfloat16"):
        check_case(make(dtype, 2, group, len_q, 70, heads, heads_kv, 32, "ragged", seed=group))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("R,G,Lq,Lk,H,Hk,D", [(1, 1, 1, 4099, 4, 1, 64), (2, 3, 5, 2050, 2, 2, 128),
                                              (1, 40, 64, 70, 1, 1, 32), (1, 9, 64, 515, 2, 1, 64)])
def test_split_axes(dtype, R, G, Lq, Lk, H, Hk, D):
    """Few rows over many keys, few keys under many rows: the long axis is split and joined."""
    say(f"attention, {dtype}, {G * Lq} rows, {Lk} keys")
    c = make(dtype, R, G, Lq, Lk, H, Hk, D, "both" if R > 1 else "none", seed=Lk)
    assert pc.pc_cross_attention_workspace(c["q"], c["k"], c["v"], backward=True) > 4 * G * Lq * H * R
    check_case(c)


def test_split_with_empty_parts():
    """Splits that hold no attended key, beside splits that do; and a state without any."""
    torch, dev = torch_dev()
    c = make("bfloat16", 3, 1, 2, 3000, 2, 2, 64, "none", seed=1)
    assert pc.pc_cross_attention_workspace(c["q"], c["k"], c["v"]) > 0
    m = torch.zeros(3, 3000, dtype=torch.uint8)
    m[0, 2900] = 1
    m[1, 5:9] = 1
    c["key_mask"] = m.to(dev)
    check_case(c)


@pytest.mark.parametrize("dtype,dim", [("float32", 40), ("bfloat16", 40), ("bfloat16", 128)])
@pytest.mark.parametrize("len_k", [600, 1300, 9000])
def test_two_to_dozens_of_parts(dtype, dim, len_k):
    """Every way the parts of a row are shared out: all attended, two keys far apart, one key, none."""
    torch, dev = torch_dev()
    say(f"attention, {dtype}, heads of {dim}, {len_k} keys in parts")
    c = make(dtype, 4, 1, 3, len_k, 3, 1, dim, "none", seed=len_k)
    m = torch.zeros(4, len_k, dtype=torch.uint8)
    m[0] = 1
    m[1, 7] = m[1, len_k - 2] = 1
    m[2, len_k // 2] = 1
    c["key_mask"] = m.to(dev)
    check_case(c)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("group,len_q,heads,heads_kv,len_k", [
    (1, 1, 1, 1, 129), (1, 33, 2, 1, 128), (2, 31, 6, 2, 200), (9, 64, 4, 4, 70), (5, 7, 5, 1, 300)])
def test_rows_of_wide_heads(dtype, group, len_q, heads, heads_kv, len_k):
    for dim in (96, 120, 128):
        say(f"attention, {dtype}, heads of {dim}, group {group}, {len_q} tokens, heads {heads}/{heads_kv}, {len_k} keys")
        check_case(make(dtype, 2, group, len_q, len_k, heads, heads_kv, dim, "both", seed=len_k))


def test_lengths_outside_their_range_are_taken_in():
    torch, dev = torch_dev()
    c = make("float32", 3, 2, 5, 40, 2, 2, 32, "none")
    c["kv_len"] = torch.tensor([-3, 1000, 7], dtype=torch.int32, device=dev)
    say("attention, kv_len below 0 and above len_k")
    u, up, ap = UNIT["float32"]
    keep = att.attended(3, 40, [0, 40, 7])
    q, k, v, g = (f64(c[n]) for n in ("q", "k", "v", "dout"))
    b = att.error_bounds(q, k, v, g, keep, c["scale"], u, up, ap)
    out, lse = forward(c)
    check("out", out, att.forward(q, k, v, keep, c["scale"])[0], b[0])
    for n, got, w, t in zip("qkv", backward(c, out, lse), att.backward(q, k, v, g, keep, c["scale"]), b[1:]):
        check("d" + n, got, w, t)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("len_k", [50, 200, 3000])
def test_unattended_places_hold_anything(dtype, len_k):
    """NaN and infinities at places that are not attended change no bit."""
    torch, dev = torch_dev()
    say(f"attention, {dtype}, {len_k} keys, NaN in masked places")
    c = make(dtype, 3, 2, 9, len_k, 2, 1, 64, "both", seed=4)
    out, lse = forward(c)
    grads = backward(c, out, lse)
    off = ~torch.from_numpy(keep_of(c)).to(dev)
    for n, bad in (("k", float("nan")), ("v", float("inf")), ("k", -float("inf")), ("v", float("nan"))):
        c[n] = torch.where(off[:, :, None, None], torch.full_like(c[n], bad), c[n])
        again, lse2 = forward(c)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
        assert all(torch.equal(a, b) for a, b in zip(backward(c, out, lse), grads))


def test_inputs_that_are_not_finite():
    """NaN stays in the rows that meet it; keys whose scores are -inf get no weight beside finite ones."""
    torch, dev = torch_dev()
    say("attention, NaN and infinite inputs")
    c = make("bfloat16", 2, 2, 40, 100, 2, 2, 64, "none", seed=5)
    clean, _ = forward(c)
    c["q"][1, 7, 0, 3] = float("nan")
    out, _ = forward(c)
    assert torch.isnan(out[1, 7, 0]).all()
    out[1, 7, 0] = clean[1, 7, 0]
    assert torch.equal(out, clean)
    c = make("float32", 1, 1, 3, 64, 1, 1, 32, "none", seed=6)
    c["q"].abs_()
    c["k"][0, 5] = -float("inf")
    out, _ = forward(c)
    c["key_mask"] = torch.ones(1, 64, dtype=torch.uint8, device=dev)
    c["key_mask"][0, 5] = 0
    want, _ = forward(c)
    assert torch.equal(out, want)
    c["key_mask"], c["k"][:] = None, -float("inf")          # no finite score at all: the softmax has no value
    out, _ = forward(c)
    assert torch.isnan(out).all()


def test_large_scores():
    """Scores of thousands: nothing overflows, the largest takes all."""
    say("attention, scores of thousands")
    for dtype in ("float32", "float16"):
        check_case(make(dtype, 2, 2, 33, 90, 2, 2, 64, "ragged", seed=8, amp=20.0))


def test_strided_views():
    """Keys and values as halves of one projection, queries and gradients with heads before tokens, one state broadcast."""
    torch, dev = torch_dev()
    say("attention, strided inputs and outputs")
    for dtype in ("float32", "bfloat16"):
        c = make(dtype, 4, 2, 37, 90, 4, 2, 40, "both", seed=9)
        out, lse = forward(c)
        grads = backward(c, out, lse)
        s = dict(c)
        kv = torch.stack((c["k"], c["v"]), dim=2)
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        swap = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
        s["q"], s["dout"] = swap(c["q"]), swap(c["dout"])
        wide = torch.full((8, 37, 4, 64), 3.0, dtype=c["q"].dtype, device=dev)
        pc.pc_cross_attention(s["q"], s["k"], s["v"], wide[..., :40], lse, s["kv_len"], s["key_mask"], s["scale"])
        assert torch.equal(wide[..., :40], out) and bool((wide[..., 40:] == 3.0).all())
        dkv = torch.full_like(kv, 7.0)
        dq = swap(torch.full_like(c["q"], 7.0))
        pc.pc_cross_attention_backward(s["q"], s["k"], s["v"], wide[..., :40], lse, s["dout"], dq, dkv[:, :, 0],
                                       dkv[:, :, 1], s["kv_len"], s["key_mask"], s["scale"])
        assert torch.equal(dq, grads[0]) and torch.equal(dkv[:, :, 0], grads[1]) and torch.equal(dkv[:, :, 1], grads[2])
        # one null state for all regions, read in place
        c["kv_len"] = c["key_mask"] = None
        b = dict(c, k=c["k"][:1].expand(4, -1, -1, -1), v=c["v"][:1].expand(4, -1, -1, -1))
        r = dict(c, k=b["k"].contiguous(), v=b["v"].contiguous())
        assert torch.equal(forward(b)[0], forward(r)[0])


def test_offsets_past_32_bits():
    """Encoder states that lie 2^31 and more elements apart in one long buffer, and such output rows."""
    torch, dev = torch_dev()
    say("attention, offsets past 2^31 elements")
    c = make("bfloat16", 2, 2, 9, 70, 2, 2, 64, "none", seed=10)
    want, _ = forward(c)
    gap = (1 << 31) + 4096
    buf = torch.zeros(gap + 70 * 2 * 64, dtype=torch.bfloat16, device=dev)
    views = []
    for n in "kv":
        view = buf.as_strided((2, 70, 2, 64), (gap, 128, 64, 1))
        view.copy_(c[n])
        views.append(view)
        got, _ = forward(dict(c, **{n: view}))
        assert torch.equal(got, want)
    wide = buf.as_strided((4, 9, 2, 64), (gap // 4 // 8 * 8, 128, 64, 1))   # batch 3 starts past 1.6e9 elements
    far = buf.as_strided((4, 9, 2, 64), (gap // 3 // 8 * 8, 128, 64, 1))    # batch 3 past 2^31
    for view in (wide, far):
        pc.pc_cross_attention(c["q"], c["k"], c["v"], view, scale=c["scale"])
        assert torch.equal(view, want)


def test_empty_axes():
    torch, dev = torch_dev()
    say("attention, axes of no entries")
    z = lambda *s: torch.zeros(*s, device=dev)  # noqa: E731
    out, lse = torch.full((4, 3, 2, 32), 7.0, device=dev), torch.full((4, 3, 2), 7.0, device=dev)
    pc.pc_cross_attention(z(4, 3, 2, 32), z(2, 0, 2, 32), z(2, 0, 2, 32), out, lse)
    assert not out.any() and bool(torch.isneginf(lse).all())
    dq, none = torch.full_like(out, 7.0), z(2, 0, 2, 32)
    pc.pc_cross_attention_backward(z(4, 3, 2, 32), none, none, out, lse, out, dq, none, none)
    assert not dq.any()
    pc.pc_cross_attention(z(0, 3, 2, 32), z(0, 5, 2, 32), z(0, 5, 2, 32), z(0, 3, 2, 32))
    q = z(4, 0, 2, 32)
    pc.pc_cross_attention(q, z(2, 5, 2, 32), z(2, 5, 2, 32), z(4, 0, 2, 32))
    dk, dv = (torch.full((2, 5, 2, 32), 7.0, device=dev) for _ in range(2))
    pc.pc_cross_attention_backward(q, z(2, 5, 2, 32), z(2, 5, 2, 32), q, z(4, 0, 2), q, q, dk, dv)
    assert not dk.any() and not dv.any()


def test_gradients_against_differences():
    """Directional derivatives of the kernel's own forward in float32.  With h = 2^-5 the central difference is off by
    h^2 / 6 times the third derivative (here below 40 of the scale of f'), the outputs' rounding by 2^-22 |f| / h."""
    torch, dev = torch_dev()
    say("attention, gradients against central differences")
    c = make("float32", 2, 2, 6, 40, 2, 1, 32, "both", seed=11)
    c["kv_len"] = None
    out, lse = forward(c)
    grads = dict(zip("qkv", backward(c, out, lse)))
    gen = torch.Generator().manual_seed(3)
    for n in "qkv":
        u = torch.randn(c[n].shape, generator=gen).to(dev)
        u /= u.norm()
        h = 2.0 ** -5
        f = []
        for s in (1.0, -1.0):
            o, _ = forward(dict(c, **{n: c[n] + s * h * u}))
            f.append((o.double() * c["dout"].double()).sum().item())
        want = (grads[n].double() * u.double()).sum().item()
        size = grads[n].double().norm().item()
        assert abs((f[0] - f[1]) / (2 * h) - want) <= h * h / 6 * 40 * size + 2.0 ** -22 * (out.norm() * c["dout"].norm()).item() / h


def test_runs_are_identical_in_slices_streams_and_graphs():
    """Repeated, cut into small dispatches, on another stream and replayed from a graph: the same bits."""
    torch, dev = torch_dev()
    say("attention, repeated / sliced / side stream / graph")
    c = make("bfloat16", 2, 5, 64, 600, 4, 2, 64, "both", seed=12)
    out, lse = forward(c)
    grads = backward(c, out, lse)

    def same(o, l, g):
        return torch.equal(o, out) and torch.equal(l, lse) and all(torch.equal(x, y) for x, y in zip(g, grads))

    o, l = forward(c)
    assert same(o, l, backward(c, o, l))
    pc.pc_set_max_dispatch_items(1024)
    try:
        o, l = forward(c)
        assert same(o, l, backward(c, o, l))
    finally:
        pc.pc_set_max_dispatch_items(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, l = forward(c)
        g = backward(c, o, l)
    torch.cuda.current_stream().wait_stream(side)
    assert same(o, l, g)
    ws = torch.empty(pc.pc_cross_attention_workspace(c["q"], c["k"], c["v"], backward=True), dtype=torch.uint8, device=dev)
    wf = torch.empty(max(16, pc.pc_cross_attention_workspace(c["q"], c["k"], c["v"])), dtype=torch.uint8, device=dev)
    o, l = torch.empty_like(out), torch.empty_like(lse)
    g = [torch.empty_like(x) for x in grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pc.pc_cross_attention(c["q"], c["k"], c["v"], o, l, c["kv_len"], c["key_mask"], c["scale"], wf)
        pc.pc_cross_attention_backward(c["q"], c["k"], c["v"], o, l, c["dout"], *g, c["kv_len"], c["key_mask"], c["scale"], ws)
    for n in range(3):
        for t in (o, l, *g):
            t.fill_(float(n))
        graph.replay()
        torch.cuda.synchronize()
        assert same(o, l, g), f"replay {n}"


def test_binding_refuses():
    torch, dev = torch_dev()
    say("attention, refusals of the binding")
    c = make("bfloat16", 2, 2, 5, 40, 4, 2, 64, "none")
    q, k, v = c["q"], c["k"], c["v"]
    out = torch.empty_like(q)
    bad = [
        lambda: pc.pc_cross_attention(q, k, v, out.float()),
        lambda: pc.pc_cross_attention(q.cpu(), k, v, out),
        lambda: pc.pc_cross_attention(q[:3], k, v, out[:3]),
        lambda: pc.pc_cross_attention(q, k, v[:, :30], out),
        lambda: pc.pc_cross_attention(q, k[..., :32], v[..., :32], out),
        lambda: pc.pc_cross_attention(q, k, v, out, key_mask=torch.ones(2, 39, dtype=torch.uint8, device=dev)),
        lambda: pc.pc_cross_attention(q, k, v, out, kv_len=torch.ones(2, dtype=torch.int64, device=dev)),
        lambda: pc.pc_cross_attention(q.double(), k.double(), v.double(), out.double()),
        lambda: pc.pc_cross_attention(q, k, v, out, lse=torch.empty(4, 4, 5, device=dev)),
        lambda: pc.pc_cross_attention(q, k, v, torch.empty(4, 5, 64, 4, dtype=q.dtype, device=dev).transpose(2, 3)),
        lambda: pc.pc_cross_attention_backward(q, k, v, out, None, out, out, k, v),
        lambda: pc.pc_cross_attention(q[0], k, v, out),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    refused = [
        lambda: pc.pc_cross_attention(q, k, v, out, scale=0.0),
        lambda: pc.pc_cross_attention(q[..., :20], k[..., :20], v[..., :20], out[..., :20]),
        lambda: pc.pc_cross_attention(q, k, v, out[:1].expand(4, -1, -1, -1)),
        lambda: pc.pc_cross_attention(q[..., 4:36], k[..., :32], v[..., :32], out[..., :32]),
        lambda: pc.pc_cross_attention(q[:, :, :3], k, v, out[:, :, :3]),
        lambda: pc.pc_cross_attention_backward(q, k, v, out, torch.empty(4, 5, 4, device=dev), out, q.clone(), k.clone(),
                                               v.clone(), workspace=torch.empty(16, dtype=torch.uint8, device=dev)),
    ]
    for f in refused:
        with pytest.raises(pc.PCError):
            f()


def test_binding_names_a_missing_tensor():
    torch, dev = torch_dev()
    say("attention, a tensor that is None")
    c = make("bfloat16", 2, 2, 5, 40, 4, 2, 64, "none")
    q, k, v = c["q"], c["k"], c["v"]
    lse = torch.empty(4, 5, 4, device=dev)
    for f, name in ((lambda: pc.pc_cross_attention(q, k, v, None), "out"),
                    (lambda: pc.pc_cross_attention_backward(q, k, v, q.clone(), lse, None, q.clone(), k.clone(), v.clone()), "dout")):
        with pytest.raises(ValueError, match=f"^{name} is required"):
            f()
