"""Timed cases of the denoiser's operators: cross attention of a map's tokens to its region's encoder
states, and the norm of queries and keys per head with the position rotation in the same pass, each
forward and with its gradients.

`own` chooses the side: False computes the operators in their plain form (elementary torch operations
in float32, rounded once at the end), True calls the library's entry points.  Cases are sized after the
workloads of this repository: 64-bead tiles at stride 52, several trajectories and guidance weights that
share one region's conditioning, chains of 32 tiles.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

BEADS, STRIDE = 64, 52
DTYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
EPS = 1e-6
BASE = 10000.0


def _attend(name, **kw):
    c = {"name": name, "op": "attend", "train": False, "dtype": "bfloat16", "regions": 1, "group": 1, "len_q": BEADS,
         "len_k": 128, "heads": 8, "heads_kv": 8, "dim": 64, "mask": "none"}
    c.update(kw)
    return c


def _norm(name, **kw):
    c = {"name": name, "op": "norm", "train": False, "dtype": "bfloat16", "regions": 1, "group": 1, "len_q": BEADS,
         "len_k": 128, "heads": 8, "heads_kv": 8, "dim": 64, "rot": 64, "interleaved": False}
    c.update(kw)
    return c


def listed():
    return [
        # One region sampled with 8 trajectories x 2 guidance weights: the smallest call, where latency counts.
        _attend("attend_one_region", group=16, len_k=64, heads=4, heads_kv=4),
        # One query token per region against a long conditioning track (a pooled token read out of it): few
        # rows, all the time is reading the states once.
        _attend("attend_single_token", regions=16, len_q=1, len_k=16384, heads=32, heads_kv=8, dim=128,
                mask="ragged"),
        # float32 network of a float32 sampler, an odd track length, bins that could not be mapped masked out.
        _attend("attend_holes_float32", dtype="float32", regions=26, group=20, len_k=333, heads=4, heads_kv=4,
                mask="holes"),
        # A chain of 32 tiles, 256 trajectories x 2 weights, each tile reading its own 512 states: the largest.
        _attend("attend_chain", regions=32, group=512, len_k=512),
        # Wide heads, queries sharing key heads, a long odd track in half precision.
        _attend("attend_long_track", dtype="float16", regions=2, group=64, len_k=4097, heads=16, heads_kv=4, dim=128),
        # Training step of one small batch: latency of the three gradients.
        _attend("attend_train_small", train=True, regions=4, group=4, len_k=100, heads=4, heads_kv=4, dim=32,
                mask="ragged"),
        # Training batch over a chain's tiles, shared key heads, ragged tracks.
        _attend("attend_train_chain", train=True, regions=32, group=64, len_k=512, heads=8, heads_kv=4,
                mask="ragged"),
        # The same gradients in float32, a head size between the powers of two.
        _attend("attend_train_float32", train=True, dtype="float32", regions=8, group=16, len_k=257, heads=4,
                heads_kv=4, dim=40, mask="holes"),
        # Queries and keys of one map: the smallest call.
        _norm("norm_one_map"),
        # Queries of every map of the 32-tile chain beside each tile's keys.
        _norm("norm_chain", regions=32, group=512, len_k=512),
        # Wide heads in float32, a part of each head rotated, adjacent pairs.
        _norm("norm_partial_float32", dtype="float32", regions=26, group=20, len_k=333, dim=128, rot=64,
              interleaved=True),
        # Training: outputs, input gradients and weight gradients, shared key heads.
        _norm("norm_train", train=True, regions=32, group=64, len_k=512, heads=8, heads_kv=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges, no dearer than the largest listed one."""
    op = rng.choice(["attend", "attend", "norm"])
    while True:
        c = {"op": op, "train": rng.random() < 0.4, "dtype": rng.choice(["bfloat16", "bfloat16", "float16", "float32"]),
             "regions": _log_int(rng, 1, 64), "group": _log_int(rng, 1, 512),
             "len_q": rng.choice([1, BEADS, _log_int(rng, 2, 256)]), "len_k": _log_int(rng, 1, 16384),
             "heads_kv": rng.choice([1, 2, 4, 8]), "dim": rng.choice([32, 40, 64, 72, 96, 128])}
        c["heads"] = c["heads_kv"] * rng.choice([1, 1, 2, 4])
        q = c["regions"] * c["group"] * c["len_q"] * c["heads"]
        k = c["regions"] * c["len_k"] * c["heads_kv"]
        elements = (q + k) * c["dim"]
        if op == "attend":
            c["mask"] = rng.choice(["none", "ragged", "holes"])
            # products, float32 ones counted by their lower rate; scores of the plain form; tensors
            flops = 4.0 * q * c["len_k"] * c["dim"] * (3.5 if c["train"] else 1.0) * (8 if c["dtype"] == "float32" else 1)
            if flops > 1.0e12 or q * c["len_k"] > (6e8 if c["train"] else 3e9) or elements > 5e8:
                continue
        else:
            c["rot"] = rng.choice([r for r in (16, 32, 64, 128, c["dim"]) if r <= c["dim"] and r % 16 == 0])
            c["interleaved"] = rng.random() < 0.5
            if elements * (2.5 if c["train"] else 1) * (2 if c["dtype"] == "float32" else 1) > 5e8:
                continue
        return c


def _maps(c):
    return c["regions"] * c["group"]


def prepare(case, seed):
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev)
    gen.manual_seed(1000003 * (seed + 1) + 17)
    dt = DTYPES[case["dtype"]]
    R, B, Lq, Lk = case["regions"], _maps(case), case["len_q"], case["len_k"]
    H, Hk, D = case["heads"], case["heads_kv"], case["dim"]

    def normal(*shape, dtype=dt, scale=1.0):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).mul_(scale).to(dtype)

    s = {"case": dict(case)}
    if case["op"] == "attend":
        # Queries as a norm per head leaves them; keys and values are the two halves of one projection of
        # the encoder's states, so they arrive as strided views of it.
        s["q"] = normal(B, Lq, H, D, scale=1.5)
        kv = normal(R, Lk, 2, Hk, D)
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        s["scale"] = 1.0 / math.sqrt(D)
        s["kv_len"] = s["key_mask"] = None
        if case["mask"] == "ragged":   # tracks of different lengths
            n = torch.randint(max(1, Lk // 2), Lk + 1, (R,), generator=gen, device=dev)
            n[-1] = Lk
            s["kv_len"] = n.to(torch.int32)
        elif case["mask"] == "holes":  # unmappable bins; one region in sixteen has no usable bin
            m = torch.rand(R, Lk, generator=gen, device=dev) < 0.85
            m[7::16] = False
            s["key_mask"] = m.to(torch.uint8)
        s["out"] = torch.empty_like(s["q"])
        if case["train"]:
            s["dout"] = normal(B, Lq, H, D)
            s["lse"] = torch.empty(B, Lq, H, dtype=torch.float32, device=dev)
            s["dq"] = torch.empty_like(s["q"])
            s["dk"], s["dv"] = (torch.empty(R, Lk, Hk, D, dtype=dt, device=dev) for _ in range(2))
        return s
    s["q"], s["k"] = normal(B, Lq, H, D), normal(R, Lk, Hk, D)
    s["wq"] = 1.0 + normal(D, dtype=torch.float32, scale=0.1)
    s["wk"] = 1.0 + normal(D, dtype=torch.float32, scale=0.1)
    # Tile r starts at bead 52 r of its chain, its track at the same bin.
    start = STRIDE * torch.arange(R, device=dev)
    jitter = int(torch.randint(0, 16, (1,), generator=gen, device=dev))
    s["pos_k"] = (start[:, None] + torch.arange(Lk, device=dev) + jitter).to(torch.int32)
    s["pos_q"] = (start.repeat_interleave(case["group"])[:, None] + torch.arange(Lq, device=dev) + jitter).to(torch.int32)
    rot = case["rot"]
    s["freqs"] = BASE ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    angle = torch.arange(STRIDE * (R - 1) + max(Lq, Lk) + jitter, device=dev, dtype=torch.float64)[:, None] * \
        torch.from_numpy(s["freqs"]).to(dev)
    s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    if case["train"]:
        s["dq_out"], s["dk_out"] = normal(B, Lq, H, D), normal(R, Lk, Hk, D)
        s["dq"], s["dk"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        s["dwq"], s["dwk"] = torch.empty_like(s["wq"]), torch.empty_like(s["wk"])
    return s


# Plain forms ---------------------------------------------------------------

def _rows(t, R, Hk):
    """[B, L, H, D] -> [R, Hk, rows, D]: every query row that reads one key head of one region."""
    B, L, H, D = t.shape
    return t.view(R, B // R, L, Hk, H // Hk, D).permute(0, 3, 1, 2, 4, 5).reshape(R, Hk, -1, D)


def _unrows(t, shape, R, Hk):
    B, L, H, D = shape
    return t.view(R, Hk, B // R, L, H // Hk, D).permute(0, 2, 3, 1, 4, 5).reshape(shape)


def _attended(s):
    c = s["case"]
    keep = torch.ones(c["regions"], c["len_k"], dtype=torch.bool, device=s["q"].device)
    if s["kv_len"] is not None:
        keep = torch.arange(c["len_k"], device=keep.device)[None, :] < s["kv_len"][:, None]
    if s["key_mask"] is not None:
        keep = keep & (s["key_mask"] != 0)
    return keep


def _plain_attend(s):
    c = s["case"]
    R, Hk, dt = c["regions"], c["heads_kv"], s["q"].dtype
    q = _rows(s["q"].float(), R, Hk)
    k, v = (t.float().permute(0, 2, 1, 3).contiguous() for t in (s["k"], s["v"]))
    x = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["scale"])
    if c["mask"] != "none":
        x.masked_fill_(~_attended(s)[:, None, None, :], -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    p /= torch.where(total == 0, torch.ones_like(total), total)
    o = torch.matmul(p, v)
    out = _unrows(o, s["q"].shape, R, Hk).to(dt)
    if not c["train"]:
        return {"out": out}
    lse = _unrows(top + total.log(), s["q"].shape[:3] + (1,), R, Hk).squeeze(-1)
    do = _rows(s["dout"].float(), R, Hk)
    dv = torch.matmul(p.transpose(2, 3).contiguous(), do)
    ds = torch.matmul(do, v.transpose(2, 3).contiguous())
    ds -= (do * o).sum(dim=-1, keepdim=True)
    ds *= p
    ds *= s["scale"]
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), q)
    return {"out": out, "lse": lse, "dq": _unrows(dq, s["q"].shape, R, Hk).to(dt),
            "dk": dk.permute(0, 2, 1, 3).to(dt).contiguous(), "dv": dv.permute(0, 2, 1, 3).to(dt).contiguous()}


def _turn(x, cos, sin, interleaved):
    """Rotates the pairs of the first 2 * cos.shape[-1] values of each head; cos and sin are [B, L, 1, rot/2]."""
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, w), dim=-1).flatten(-2) if interleaved else torch.cat((u, w), dim=-1)
    return torch.cat((turned, x[..., 2 * half:]), dim=-1)


def _plain_norm(s, which):
    c = s["case"]
    x, w, pos = s[which].float(), s["w" + which], s["pos_" + which].long()
    cos, sin = s["cos"][pos][:, :, None, :], s["sin"][pos][:, :, None, :]
    rstd = torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS)
    hat = x * rstd
    r = {which + "_out": _turn(hat * w, cos, sin, c["interleaved"]).to(s[which].dtype)}
    if c["train"]:
        g = _turn(s["d" + which + "_out"].float(), cos, -sin, c["interleaved"])
        r["dw" + which] = (g * hat).sum(dim=(0, 1, 2))
        g = g * w
        r["d" + which] = (rstd * (g - hat * (g * hat).mean(dim=-1, keepdim=True))).to(s[which].dtype)
    return r


# ---------------------------------------------------------------------------

def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain_attend(s) if c["op"] == "attend" else {**_plain_norm(s, "q"), **_plain_norm(s, "k")}
    import tiled_genome_diffusion_amd as pc

    if c["op"] == "attend":
        masks = {"kv_len": s["kv_len"], "key_mask": s["key_mask"], "scale": s["scale"]}
        if not c["train"]:
            pc.pc_cross_attention(s["q"], s["k"], s["v"], s["out"], **masks)
            return {"out": s["out"]}
        pc.pc_cross_attention(s["q"], s["k"], s["v"], s["out"], s["lse"], **masks)
        pc.pc_cross_attention_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["dq"], s["dk"], s["dv"],
                                       **masks)
        return {n: s[n] for n in ("out", "lse", "dq", "dk", "dv")}
    sides = (s["q"], s["k"], s["wq"], s["wk"], s["pos_q"], s["pos_k"], s["freqs"])
    pc.pc_qk_norm_rope(*sides, s["q_out"], s["k_out"], eps=EPS, interleaved=c["interleaved"])
    if not c["train"]:
        return {n: s[n] for n in ("q_out", "k_out")}
    pc.pc_qk_norm_rope_backward(*sides, s["dq_out"], s["dk_out"], s["dq"], s["dk"], s["dwq"], s["dwk"], eps=EPS,
                                interleaved=c["interleaved"])
    return {n: s[n] for n in ("q_out", "k_out", "dq", "dk", "dwq", "dwk")}


def work(case):
    c = case
    size = 4 if c["dtype"] == "float32" else 2
    q = _maps(c) * c["len_q"] * c["heads"] * c["dim"]
    k = c["regions"] * c["len_k"] * c["heads_kv"] * c["dim"]
    rows = _maps(c) * c["len_q"] * c["heads"]
    if c["op"] == "norm":
        tokens = _maps(c) * c["len_q"] + c["regions"] * c["len_k"]
        passes = 4 if c["train"] else 2   # x read, y written; dy read, dx written
        return {"bytes": passes * size * (q + k) + 4 * tokens, "flops": (30 if c["train"] else 10) * (q + k)}
    share = {"none": 1.0, "ragged": 0.75, "holes": 0.85}[c["mask"]]   # of the states that are attended
    pairs = share * rows * c["len_k"] * c["dim"]
    if not c["train"]:   # q, k, v read; out written; q k^T and p v
        return {"bytes": size * (2 * q + 2 * share * k), "flops": 4 * pairs}
    # q, k, v, dout read; out, lse, dq, dk, dv written; the forward's two products and the gradients' five
    return {"bytes": size * (4 * q + (2 * share + 2) * k) + 4 * rows, "flops": 14 * pairs}


# Definitions in 64 bits ----------------------------------------------------

def _exact_attend(s):
    c = s["case"]
    G, H, Hk, train = c["group"], c["heads"], c["heads_kv"], c["train"]
    names = ("out", "lse", "dq", "dk", "dv") if train else ("out",)
    whole = {n: torch.zeros(s[n].shape, dtype=torch.float64, device=s["q"].device) for n in names}
    for r in range(c["regions"]):
        at = torch.arange(c["len_k"], device=s["q"].device)
        if s["kv_len"] is not None:
            at = at[: int(s["kv_len"][r])]
        if s["key_mask"] is not None:
            at = at[s["key_mask"][r, at] != 0]
        if train:
            whole["lse"][r * G:(r + 1) * G] = -math.inf
        if at.numel() == 0:
            continue
        for h in range(H):
            sl = slice(r * G, (r + 1) * G)
            q = s["q"][sl, :, h].double().requires_grad_(train)
            k = s["k"][r, at, h * Hk // H].double().requires_grad_(train)
            v = s["v"][r, at, h * Hk // H].double().requires_grad_(train)
            with torch.set_grad_enabled(train):
                x = torch.matmul(q.flatten(0, 1), k.t()) * s["scale"]
                lse = torch.logsumexp(x, dim=-1)
                o = torch.matmul((x - lse[:, None]).exp(), v).view(q.shape)
            whole["out"][sl, :, h] = o.detach()
            if train:
                o.backward(s["dout"][sl, :, h].double())
                whole["lse"][sl, :, h] = lse.detach().view(q.shape[:2])
                whole["dq"][sl, :, h] = q.grad
                whole["dk"][r, at, h * Hk // H] += k.grad
                whole["dv"][r, at, h * Hk // H] += v.grad
    return whole


def _exact_norm(s, which):
    c = s["case"]
    half = c["rot"] // 2
    train = c["train"]
    x = s[which].double().requires_grad_(train)
    w = s["w" + which].double().requires_grad_(train)
    a = s["pos_" + which].double()[:, :, None] * torch.from_numpy(s["freqs"]).to(x.device)
    z = torch.polar(torch.ones_like(a), a)[:, :, None, :]   # one unit complex number per pair
    with torch.set_grad_enabled(train):
        y = x / torch.sqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * w
        first = y[..., : 2 * half]
        pairs = first.unflatten(-1, (half, 2)) if c["interleaved"] else first.unflatten(-1, (2, half)).transpose(-1, -2)
        turned = torch.view_as_real(torch.complex(pairs[..., 0], pairs[..., 1]) * z)
        turned = turned.flatten(-2) if c["interleaved"] else turned.transpose(-1, -2).flatten(-2)
        y = torch.cat((turned, y[..., 2 * half:]), dim=-1)
    r = {which + "_out": y.detach()}
    if train:
        y.backward(s["d" + which + "_out"].double())
        r["d" + which], r["dw" + which] = x.grad, w.grad
    return r


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(s)
    return {**_exact_norm(s, "q"), **_exact_norm(s, "k")}
