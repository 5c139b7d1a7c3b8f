"""The conditioning operators of the attention block, as measured cases: per-head norms of Q and K with the rotary
embedding in one pass (``qk``), cross attention to an encoder's states (``cross``) and attention over a shared prefix
followed by a sample's own keys (``prefix``).

``run`` computes them in elementary torch operations, or (``own``) through the framework's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
HEAD_DIMS = (32, 64, 72, 80, 96, 128)
EPS = 1e-6


# ---------------------------------------------------------------- cases
def _qk(name, n, hq, hk, d, dtype="bf16", pairing="interleaved", period=0, given=False, fused=False):
    return {"name": name, "op": "qk", "n": n, "hq": hq, "hk": hk, "d": d, "dtype": dtype, "pairing": pairing,
            "period": period, "given": given, "fused": fused}


def _cross(name, b, t, s, h, d, l, hkv=0, sets=0, dtype="bf16", layout="dense"):
    return {"name": name, "op": "cross", "b": b, "t": t, "s": s, "h": h, "hkv": hkv or h, "d": d, "l": l,
            "sets": sets or b, "dtype": dtype, "layout": layout}


def _prefix(name, b, sets, s, h, d, lp, l, hkv=0, dtype="bf16", ragged=False):
    return {"name": name, "op": "prefix", "b": b, "t": 1, "sets": sets, "s": s, "h": h, "hkv": hkv or h, "d": d,
            "lp": lp, "l": l, "dtype": dtype, "ragged": ragged}


def listed():
    return [
        # the fp32 block of 4 frames of 64 tokens: latency of a small call
        _qk("qk_tiny_fp32", 256, 2, 2, 32, "fp32", period=64),
        # 16 frames of 1200 tokens, Q and K read out of the fused projection, position = index in the frame
        _qk("qk_opensora_low", 19200, 16, 16, 72, period=1200, fused=True),
        # the 65,536-token image, halves pairing, positions given per token
        _qk("qk_image_4096px", 65536, 24, 24, 128, pairing="halves", given=True),
        # the fp32 block attending to 20 text tokens
        _cross("cross_tiny_fp32", 2, 4, 64, 2, 32, 20, dtype="fp32"),
        # a pooling query per sample over a prompt: the smallest call in bf16
        _cross("cross_one_query", 8, 1, 1, 16, 72, 300, layout="padded"),
        # the low-resolution video block with both guidance branches, prompts padded to 300 tokens
        _cross("cross_opensora_low", 2, 16, 1200, 16, 72, 300, layout="padded"),
        # the 1080p video block, prompts packed one behind the other
        _cross("cross_video_1080p", 1, 32, 8160, 16, 72, 300, layout="packed"),
        # the 65,536-token image attending to 512 text tokens under the tokenizer's mask
        _cross("cross_image_4096px", 1, 1, 65536, 24, 128, 512, layout="masked"),
        # one query per sample over long encoder states, grouped heads: the keys have to be split over the GPU
        _cross("cross_long_states", 2, 1, 1, 24, 128, 20736, hkv=8),
        # four samples of one prompt continuing two shared reference frames
        _prefix("prefix_opensora_low", 4, 1, 1200, 16, 72, 2400, 1200),
        # joint attention of an image's 4096 tokens behind its prompt's tokens
        _prefix("prefix_joint_image", 2, 2, 4096, 24, 128, 300, 4096),
        # one token per sample: 64 samples share a long prefix, each with up to 64 keys of its own
        _prefix("prefix_one_token", 64, 1, 1, 16, 72, 16384, 64, ragged=True),
    ]


MOST_BYTES, MOST_FLOPS, MOST_SCORES = 1.6e9, 2.4e11, 1.2e9


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(("qk", "cross", "cross", "prefix"))
        dtype = "fp32" if rng.random() < 0.2 else "bf16"
        hkv = rng.randint(1, 8)
        h = hkv * rng.choice((1, 1, 1, 2, 3))
        if op == "qk":
            n = _log(rng, 1, 65536)
            c = _qk("", n, rng.randint(1, 24), rng.randint(1, 24), rng.choice(HEAD_DIMS), dtype,
                    rng.choice(("interleaved", "halves")), rng.choice((0, max(1, n // rng.randint(1, 16)))),
                    rng.random() < 0.4, rng.random() < 0.4)
        elif op == "cross":
            b = rng.randint(1, 8)
            few = rng.random() < 0.3
            s = rng.randint(1, 64) if few else _log(rng, 64, 65536)
            l = _log(rng, 64, 20736) if few else _log(rng, 1, 600)
            layout = rng.choice(("dense", "padded", "packed", "masked"))
            c = _cross("", b, rng.choice((1, 1, 2, 5, 16)), s, h, rng.choice(HEAD_DIMS), l, hkv,
                       1 if rng.random() < 0.2 else b, dtype, layout)
        else:
            few = rng.random() < 0.4
            sets = rng.randint(1, 4)
            c = _prefix("", sets * (_log(rng, 1, 32) if few else rng.randint(1, 4)), sets,
                        rng.randint(1, 16) if few else _log(rng, 64, 4096), h, rng.choice(HEAD_DIMS),
                        _log(rng, 1, 16384 if few else 4096), _log(rng, 1, 256 if few else 4096), hkv, dtype,
                        rng.random() < 0.5)
        del c["name"]
        w = work(c)
        scores = 0 if op == "qk" else c["b"] * c["t"] * c["s"] * c["h"] * (c["l"] + c.get("lp", 0))
        limit = 0.1 if dtype == "fp32" and op != "qk" else 1.0
        if w["bytes"] <= limit * MOST_BYTES and w["flops"] <= limit * MOST_FLOPS and scores <= limit * MOST_SCORES:
            return c


# ---------------------------------------------------------------- inputs
def _lens(n, most, seed):
    """Lengths in [1, most], the first one whole (a prompt that fills its place)."""
    g = torch.Generator().manual_seed(7919 * seed + 13)
    x = torch.randint(1, most + 1, (n,), generator=g, dtype=torch.int32)
    x[0] = most
    return x


def prepare(case, seed):
    c = case
    dt = DTYPES[c["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device="cuda", dtype=torch.float32, generator=gen).to(dt)

    st = {"case": dict(c)}
    if c["op"] == "qk":
        n, hq, hk, d = c["n"], c["hq"], c["hk"], c["d"]
        if c["fused"]:                          # rows [Q | K | V] of one projection
            x = normal(n, hq + 2 * hk, d)
            st["q"], st["k"] = x[:, :hq], x[:, hq:hq + hk]
        else:
            st["q"], st["k"] = normal(n, hq, d), normal(n, hk, d)
        st["q_gamma"] = 1 + 0.1 * torch.randn(d, device="cuda", generator=gen)
        st["k_gamma"] = 1 + 0.1 * torch.randn(d, device="cuda", generator=gen)
        n_pos = c["period"] or n
        ang = torch.arange(n_pos, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
        st["table"] = torch.stack((ang.cos(), ang.sin()), -1).float().contiguous()
        st["positions"] = None
        if c["given"]:                          # e.g. the scan order of an image of another aspect; -1: a text token
            st["positions"] = torch.randint(-1, n_pos, (n,), device="cuda", generator=gen).int()
        st["q_out"] = torch.empty(n, hq, d, device="cuda", dtype=dt)
        st["k_out"] = torch.empty(n, hk, d, device="cuda", dtype=dt)
        return st
    b, s, h, hkv, d, l, sets = c["b"], c["s"], c["h"], c["hkv"], c["d"], c["l"], c["sets"]
    st["q"] = normal(b, c["t"], s, h, d)
    st["o"] = torch.empty_like(st["q"])
    if c["op"] == "cross":
        layout = c["layout"]
        st["len"] = st["offsets"] = st["mask"] = None
        if layout == "packed":
            lens = _lens(sets, l, seed)
            off = torch.zeros(sets + 1, dtype=torch.int32)
            off[1:] = lens.cumsum(0)
            st["offsets"] = off.cuda()
            kv = normal(int(off[-1]), 2, hkv, d)
            st["k"], st["v"] = kv[:, 0], kv[:, 1]
        else:
            kv = normal(sets, l, 2, hkv, d)     # one projection gives both
            st["k"], st["v"] = kv[:, :, 0], kv[:, :, 1]
            if layout == "padded":
                st["len"] = _lens(sets, l, seed).cuda()
            elif layout == "masked":
                keep = torch.rand(sets, l, device="cuda", generator=gen) < 0.9
                keep &= torch.arange(l, device="cuda") < _lens(sets, l, seed).cuda()[:, None]
                keep[:, 0] = True
                st["mask"] = keep.to(torch.uint8)
    else:
        st["kp"], st["vp"] = normal(sets, c["lp"], hkv, d), normal(sets, c["lp"], hkv, d)
        st["k"], st["v"] = normal(b, l, hkv, d), normal(b, l, hkv, d)
        st["len"] = _lens(b, l, seed).cuda() if c["ragged"] else None
    return st


# ---------------------------------------------------------------- one pass
def _plain_norm(x, gamma, table, pos, pairing):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma
    turned = (pos >= 0) & (pos < table.shape[0])
    cs = table[pos.clamp(0, table.shape[0] - 1)]
    cos = torch.where(turned[:, None], cs[..., 0], 1.0)[:, None]
    sin = torch.where(turned[:, None], cs[..., 1], 0.0)[:, None]
    if pairing == "interleaved":
        a, b = y[..., 0::2], y[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    a, b = y.chunk(2, -1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _plain_attention(q, k, v, keep):
    """q [B,T,S,H,D]; k, v [B,L,Hkv,D]; keep [B,L] of truth values or None."""
    b, t, s, h, d = q.shape
    hkv = k.shape[2]
    qh = q.float().reshape(b, t * s, hkv, h // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    kh, vh = k.float().permute(0, 2, 3, 1), v.float().transpose(1, 2)
    x = qh @ kh * (1.0 / math.sqrt(d))
    if keep is not None:
        x = x.masked_fill(~keep[:, None, None, :], -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp_()
    o = (x @ vh) / x.sum(-1, keepdim=True)
    return o.reshape(b, hkv, h // hkv, t * s, d).permute(0, 3, 1, 2, 4).reshape(b, t, s, h, d).to(q.dtype)


def _plain(st):
    c = st["case"]
    if c["op"] == "qk":
        pos = st["positions"]
        if pos is None:
            pos = torch.arange(c["n"], device="cuda") % (c["period"] or c["n"])
        pos = pos.long()
        return {n: _plain_norm(st[n], st[n + "_gamma"], st["table"], pos, c["pairing"]).to(st[n].dtype) for n in "qk"}
    if c["op"] == "cross":
        k, v, keep = st["k"], st["v"], None
        at = torch.arange(c["l"], device="cuda")
        if st["offsets"] is not None:           # packed rows to padded ones
            off = st["offsets"].long()
            keep = at < (off[1:] - off[:-1])[:, None]
            rows = (off[:-1, None] + at).clamp(max=k.shape[0] - 1)
            k, v = k[rows], v[rows]
        elif st["len"] is not None:
            keep = at < st["len"][:, None]
        elif st["mask"] is not None:
            keep = st["mask"] != 0
    else:
        each = c["b"] // c["sets"]
        k = torch.cat((st["kp"].repeat_interleave(each, 0), st["k"]), 1)
        v = torch.cat((st["vp"].repeat_interleave(each, 0), st["v"]), 1)
        keep = None
        if st["len"] is not None:
            at = torch.arange(c["lp"] + c["l"], device="cuda")
            keep = at < c["lp"] + st["len"][:, None]
    if k.shape[0] != c["b"]:
        each = c["b"] // k.shape[0]
        k, v = k.repeat_interleave(each, 0), v.repeat_interleave(each, 0)
        keep = None if keep is None else keep.repeat_interleave(each, 0)
    return _plain_attention(st["q"], k, v, keep)


def _own(st):
    import sequence_parallelism_st_b200 as lib
    c = st["case"]
    if c["op"] == "qk":
        lib.st_qk_norm_rope(st["q"], st["k"], st["q_out"], st["k_out"], st["q_gamma"], st["k_gamma"], EPS,
                            rope_table=st["table"], positions=st["positions"], pos_period=c["period"],
                            pairing=c["pairing"])
        return {"q": st["q_out"], "k": st["k_out"]}
    if c["op"] == "cross":
        kw = dict(kv_len=st["len"], kv_offsets=st["offsets"], kv_mask=st["mask"])
        if st["offsets"] is not None:
            kw["max_len"] = c["l"]
        if "workspace" not in st:
            n = lib.st_attn_cross_workspace_bytes(st["q"], st["k"], **kw)
            st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        lib.st_attn_cross(st["q"], st["k"], st["v"], st["o"], workspace=st["workspace"], **kw)
        return st["o"]
    if "workspace" not in st:
        n = lib.st_attn_prefix_workspace_bytes(st["q"], st["kp"], st["k"], kv_len=st["len"])
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    lib.st_attn_prefix(st["q"], st["kp"], st["vp"], st["k"], st["v"], st["o"], kv_len=st["len"],
                       workspace=st["workspace"])
    return st["o"]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    e = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "qk":
        n, heads, d = c["n"], c["hq"] + c["hk"], c["d"]
        n_pos = c["period"] or n
        return {"bytes": 2 * n * heads * d * e + n_pos * d * 4 + (4 * n if c["given"] else 0),
                "flops": 10 * n * heads * d}
    rows = c["b"] * c["t"] * c["s"] * c["h"]
    if c["op"] == "cross":
        # a mean length: lengths are drawn with the seed (the first set is whole)
        keys = c["l"] if c["layout"] == "dense" else (c["l"] + (c["sets"] - 1) * (c["l"] + 1) / 2) / c["sets"]
        held = c["sets"] * keys
    else:
        own_keys = (c["l"] + (c["b"] - 1) * (c["l"] + 1) / 2) / c["b"] if c["ragged"] else c["l"]
        keys = c["lp"] + own_keys
        held = c["sets"] * c["lp"] + c["b"] * own_keys
    return {"bytes": 2 * rows * c["d"] * e + 2 * held * c["hkv"] * c["d"] * e, "flops": 4 * rows * keys * c["d"]}


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_rows(q, ks, vs, group):
    """Rows of one sample: q [R,H,D] against the keys ks [L,Hkv,D] that count."""
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    if ks.shape[0] == 0:
        return out
    step = max(1, 200_000_000 // ks.shape[0])
    for h in range(q.shape[1]):
        k, v = ks[:, h // group].double(), vs[:, h // group].double()
        for r in range(0, q.shape[0], step):
            z = torch.mm(q[r:r + step, h].double(), k.t()).div_(math.sqrt(q.shape[2]))
            out[r:r + step, h] = torch.softmax(z, dim=1).mm(v)
    return out


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] == "qk":
        got = {}
        for name in "qk":
            x = st[name].double()
            y = x / ((x * x).sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * st[name + "_gamma"].double()
            z = torch.view_as_complex(st["table"].double())
            p = st["positions"]
            p = torch.arange(c["n"], device="cuda").remainder(z.shape[0]) if p is None else p.long()
            z = torch.cat((z, torch.ones_like(z[:1])))[torch.where((p < 0) | (p >= z.shape[0]), z.shape[0], p)]
            if c["pairing"] == "interleaved":
                w = torch.view_as_complex(y.unflatten(-1, (-1, 2)).contiguous()) * z[:, None]
                got[name] = torch.view_as_real(w).flatten(-2)
            else:
                w = torch.complex(y[..., :c["d"] // 2].contiguous(), y[..., c["d"] // 2:].contiguous()) * z[:, None]
                got[name] = torch.cat((w.real, w.imag), -1)
        return got
    group = c["h"] // c["hkv"]
    outs = []
    for i in range(c["b"]):
        q = st["q"][i].flatten(0, 1)
        if c["op"] == "cross":
            j = i // (c["b"] // c["sets"])
            if st["offsets"] is not None:
                a, z = int(st["offsets"][j]), int(st["offsets"][j + 1])
                k, v = st["k"][a:z], st["v"][a:z]
            else:
                k, v = st["k"][j], st["v"][j]
                if st["len"] is not None:
                    k, v = k[:int(st["len"][j])], v[:int(st["len"][j])]
                if st["mask"] is not None:
                    at = st["mask"][j].nonzero().flatten()
                    k, v = k[at], v[at]
        else:
            j = i // (c["b"] // c["sets"])
            n = c["l"] if st["len"] is None else int(st["len"][i])
            k, v = torch.cat((st["kp"][j], st["k"][i, :n])), torch.cat((st["vp"][j], st["v"][i, :n]))
        outs.append(_exact_rows(q, k, v, group).reshape(st["q"][i].shape))
    return torch.stack(outs)
