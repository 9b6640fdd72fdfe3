"""Measured cases of the 8-bit KV cache path of an uncompressed (multi-KV-head)
attention layer: per-head norm + rotation of queries and keys, append of new
tokens to the cache, attention over the cache, and eviction of whole token
blocks by their accumulated attention weight.

Cache: per sequence and KV head N slots of d E4M3 codes for K and for V and,
for every `block` consecutive slots, one exponent byte e + 127; a stored value
is code * 2^e.

`run` computes an operator from elementary torch operations (32 bits; 64 for
angles) where `own` is false, and calls the framework where it is true.
`exact` gives the definition's values in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
E_MIN, E_MAX = -110, 119        # exponents a block may have
ACT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases --
def listed():
    norm = dict(op="norm_rope", fused=True, eps=1e-6)
    cache = dict(block=64, act="bf16")
    return [
        # a decode step of four sequences deep in a long context: launch latency counts
        dict(norm, name="norm_rope decode 4", R=4, n_q=64, n_kv=8, d=128, rope=128, half=True,
             scaling="parts", pos0=1048000, act="bf16"),
        # a whole 32K prompt, the last 64 of 128 dims rotated in interleaved pairs
        dict(norm, name="norm_rope prefill 32k", R=32768, n_q=64, n_kv=8, d=128, rope=64,
             half=False, scaling="none", pos0=0, act="bf16"),
        # fp32 activations, odd token count, heads of 96 dims, linearly scaled positions
        dict(norm, name="norm_rope f32 odd", R=1537, n_q=12, n_kv=3, d=96, rope=96, half=True,
             scaling="linear", pos0=65536, act="f32"),
        # one new token for each of 32 sequences, most of them inside an open block
        dict(cache, op="append", name="append decode 32", B=32, T=1, n_kv=8, d=128, N=4096,
             len=4001, ragged=True, cut=False),
        # a 32K prompt written in one call
        dict(cache, op="append", name="append prefill 32k", B=1, T=32768, n_kv=8, d=128,
             N=32832, len=17, ragged=False, cut=False),
        # a padded batch of prompts of unlike lengths in fp32
        dict(op="append", name="append padded f32", B=5, T=777, n_kv=3, d=64, N=2048, len=301,
             ragged=True, cut=True, block=32, act="f32"),
        # one short sequence: launch latency counts
        dict(cache, op="attend", name="attend decode short", B=1, Q=1, n_q=8, n_kv=2, d=64,
             N=2048, len=1111, ragged=False, acc=False, sink=False),
        # 32 sequences of up to 64K tokens, weights accumulated for eviction
        dict(cache, op="attend", name="attend decode 32x64k", B=32, Q=1, n_q=64, n_kv=8, d=128,
             N=65536, len=65503, ragged=True, acc=True, sink=False),
        # four sequences of a million tokens with a sink logit per head
        dict(cache, op="attend", name="attend decode 4x1m", B=4, Q=1, n_q=64, n_kv=4, d=128,
             N=1048576, len=1048576, ragged=False, acc=False, sink=True),
        # a chunk of a long prompt against 32K tokens of cache
        dict(cache, op="attend", name="attend prefill 2k of 32k", B=1, Q=2048, n_q=64, n_kv=8,
             d=128, N=32768, len=32768, ragged=False, acc=False, sink=False),
        # one block over budget: a short cache after a decode period
        dict(cache, op="evict", name="evict one block", B=4, n_kv=8, d=128, N=8192, len=8000,
             ragged=False, keep=124, recent=4),
        # long prompts cut to half the blocks
        dict(cache, op="evict", name="evict half of 64k", B=8, n_kv=8, d=128, N=65536, len=65321,
             ragged=True, keep=512, recent=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attend", "attend", "evict"])
    act = rng.choice(["bf16", "bf16", "f32"])
    n_kv = rng.choice([1, 2, 3, 4, 8])
    block = rng.choice([16, 32, 64, 128])
    if op == "norm_rope":
        d = rng.choice([64, 96, 128, 256])
        rope = rng.choice([d, d // 2, 2 * rng.randint(1, d // 2)])
        return dict(op=op, R=_log(rng, 1, 16384), n_q=n_kv * rng.choice([1, 2, 4, 8]), n_kv=n_kv,
                    d=d, rope=rope, half=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "parts"]),
                    pos0=rng.choice([0, _log(rng, 1, 1 << 20)]), act=act,
                    fused=rng.random() < 0.5, eps=1e-6)
    d = rng.choice([64, 128, 128, 256])
    if op == "append":
        B = _log(rng, 1, 32)
        T = rng.choice([1, _log(rng, 1, 16384 // B)])
        n = _log(rng, 1, 65536 // B)
        return dict(op=op, B=B, T=T, n_kv=n_kv, d=d, N=-(-(n + T) // block) * block, len=n,
                    ragged=rng.random() < 0.7, cut=rng.random() < 0.5, block=block, act=act)
    if op == "evict":
        n = _log(rng, 200, 65536)
        nb = -(-n // block)
        keep = rng.randint(1, nb)
        return dict(op=op, B=_log(rng, 1, 8), n_kv=n_kv, d=d, N=(nb + rng.randint(0, 3)) * block,
                    len=n, ragged=rng.random() < 0.7, keep=keep, recent=rng.randint(1, min(keep, 8)),
                    block=block, act=act)
    g = rng.choice([1, 2, 4, 7, 8, 16])
    if rng.random() < 0.35:          # prompt chunks
        Q, B = _log(rng, 16, 1024), _log(rng, 1, 3)
        n = max(Q, _log(rng, 64, 16384))
        n = min(n, max(Q, int(1.5e9 / (B * Q * n_kv * g))))
    else:                            # decode, with a few tokens a step at most
        Q, B = rng.choice([1, 1, 1, 2, 3, 5]), _log(rng, 1, 32)
        n = _log(rng, 1, 131072)
        n = min(n, max(1, int(1e9 / (B * n_kv * d))))
    return dict(op=op, B=B, Q=Q, n_q=n_kv * g, n_kv=n_kv, d=d, N=-(-(n + rng.randint(0, 99)) // block) * block,
                len=n, ragged=rng.random() < 0.6, acc=rng.random() < 0.4, sink=rng.random() < 0.4,
                block=block, act=act)


def _lens(c):
    """Tokens in the cache of each sequence before the call; a ragged batch
    runs from len down to about half of it."""
    return [c["len"] - (b * c["len"] // (2 * c["B"]) if c["ragged"] else 0) for b in range(c["B"])]


def _news(c):
    """New tokens of each sequence; a cut (padded) batch holds fewer than T in most."""
    return [c["T"] * (c["B"] - b) // c["B"] if c["cut"] else c["T"] for b in range(c["B"])]


def work(c):
    es = 2 if c.get("act") == "bf16" else 4
    if c["op"] == "norm_rope":
        n = c["R"] * (c["n_q"] + c["n_kv"]) * c["d"]
        return {"bytes": 2 * es * n + 4 * c["R"], "flops": 8 * n}
    if c["op"] == "append":
        n = 2 * sum(_news(c)) * c["n_kv"] * c["d"]
        return {"bytes": n * (es + 1), "flops": 3 * n}
    if c["op"] == "evict":
        nb = [-(-n // c["block"]) for n in _lens(c)]
        rank = sum(nb) * c["n_kv"]
        # of the kept blocks the share that lies above the kept range moves
        move = sum(c["keep"] * (n - c["keep"]) / n for n in nb if n > c["keep"]) * c["n_kv"]
        return {"bytes": 8 * rank + 2 * move * 2 * (c["block"] * c["d"] + 1), "flops": 4 * rank}
    lens = _lens(c)
    vis = sum(max(0, n - c["Q"] + 1 + j) for n in lens for j in range(c["Q"]))
    rows = c["B"] * c["Q"] * c["n_q"] * c["d"]
    b = 2 * sum(lens) * c["n_kv"] * c["d"] + 2 * sum(-(-n // c["block"]) for n in lens) * c["n_kv"]
    b += 2 * es * rows + (8 * sum(-(-n // c["block"]) for n in lens) * c["n_kv"] if c["acc"] else 0)
    return {"bytes": b, "flops": 4 * c["d"] * c["n_q"] * vis}


# ------------------------------------------------------------------ inputs --
def _turns(c):
    """Turns per token of each pair, in 64 bits (the table a program computes once)."""
    D, base, s, L = c["rope"], 10000.0, 8.0, 131072.0
    p = torch.arange(D // 2, dtype=torch.float64)
    t = base ** (-2.0 * p / D) / (2.0 * math.pi)
    if c["scaling"] == "linear":
        t = t / s
    elif c["scaling"] == "parts":
        ramp = ((L * t - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        t = t * ((1.0 - ramp) / s + ramp)
    return t


def _mscale(c):
    return 0.1 * math.log(8.0) + 1.0 if c["scaling"] == "parts" else 1.0


def _codes(shape, g):
    """E4M3 codes of keys or values: normal, with a few large channels."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float16)
    x[..., :: 29] *= 3.0
    return (x * 56.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    act = ACT[c["act"]]

    def rnd(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    if c["op"] == "norm_rope":
        R, n_q, n_kv, d = c["R"], c["n_q"], c["n_kv"], c["d"]
        if c["fused"]:   # views of one projection's output [R][(n_q + 2 n_kv) d]
            x = rnd(R, (n_q + 2 * n_kv) * d).to(act)
            q = x[:, :n_q * d].view(R, n_q, d)
            k = x[:, n_q * d:(n_q + n_kv) * d].view(R, n_kv, d)
        else:
            q, k = rnd(R, n_q, d).to(act), rnd(R, n_kv, d).to(act)
        return dict(c=c, q=q, k=k, gq=1.0 + 0.2 * rnd(d), gk=1.0 + 0.2 * rnd(d),
                    pos=(c["pos0"] + torch.arange(R, device=DEV)).to(torch.int32),
                    turns=_turns(c).to(DEV), q_out=torch.empty(R, n_q, d, dtype=act, device=DEV),
                    k_out=torch.empty(R, n_kv, d, dtype=act, device=DEV))
    B, H, N, d, blk = c["B"], c["n_kv"], c["N"], c["d"], c["block"]
    n_tok = torch.tensor(_lens(c), dtype=torch.int32, device=DEV)
    s = dict(c=c, kc=_codes((B, H, N, d), g), vc=_codes((B, H, N, d), g))
    for name in ("k_exp", "v_exp"):
        s[name] = torch.randint(127 - 7, 127 - 4, (B, H, N // blk), generator=g, device=DEV,
                                dtype=torch.uint8)
    if c["op"] == "append":
        # the layer's K and V of the new tokens: channels of unlike size, magnitudes that drift
        T = c["T"]
        drift = 1.0 + 2.0 * torch.rand(B, T, 1, 1, generator=g, device=DEV)
        s.update(k=(rnd(B, T, H, d) * drift).to(act), v=(rnd(B, T, H, d) * drift).to(act), n_old=n_tok,
                 n_new=torch.tensor(_news(c), dtype=torch.int32, device=DEV))
    elif c["op"] == "evict":
        acc = torch.rand(B, H, N // blk, generator=g, device=DEV).log().neg() ** 3
        acc[..., ::7] = 0.0   # blocks nothing attended: ties
        s.update(acc=acc, n_tok=n_tok, n_tok_out=torch.empty_like(n_tok), acc_out=torch.empty_like(acc),
                 kept=torch.empty(B, H, c["keep"], dtype=torch.int32, device=DEV))
    else:
        Q, n_q = c["Q"], c["n_q"]
        q = (1.5 * rnd(B * Q, n_q, d)).to(act)
        n_vis = (n_tok[:, None] - Q + 1 + torch.arange(Q, device=DEV)).clamp_(min=0).to(torch.int32)
        s.update(q=q, n_vis=n_vis.reshape(-1).contiguous(), out=torch.empty_like(q),
                 sink=rnd(n_q) if c["sink"] else None,
                 acc=torch.rand(B, H, N // blk, generator=g, device=DEV) if c["acc"] else None)
    return s


# ------------------------------------------------------------- plain forms --
def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _pow2(e):
    return torch.exp2(e.float())


def _plain_norm_rope(s):
    c = s["c"]
    D, off = c["rope"], c["d"] - c["rope"]
    turn = s["pos"].double()[:, None] * s["turns"]
    ang = (turn - turn.round()) * (2.0 * math.pi)
    cs, sn = ((f(ang) * _mscale(c)).float()[:, None, :] for f in (torch.cos, torch.sin))

    def one(x, gain):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + c["eps"]) * gain
        r = x[..., off:]
        a, b = (r[..., : D // 2], r[..., D // 2:]) if c["half"] else (r[..., 0::2], r[..., 1::2])
        u, w = a * cs - b * sn, a * sn + b * cs
        r = torch.cat([u, w], -1) if c["half"] else torch.stack([u, w], -1).flatten(-2)
        return torch.cat([x[..., :off], r], -1).to(ACT[c["act"]])

    return [one(s["q"], s["gq"]), one(s["k"], s["gk"])]


def _plain_store(x, n_old, n_new, codes, exps, blk):
    B, T, H, d = x.shape
    nbt = min((T + blk - 2) // blk + 1, codes.shape[2] // blk)   # blocks a sequence can touch
    first = (n_old // blk).long()
    blocks = first[:, None] + torch.arange(nbt, device=DEV)                # [B, nbt]
    inside = blocks < exps.shape[2]
    blocks = blocks.clamp(max=exps.shape[2] - 1)
    slot = blocks[:, :, None] * blk + torch.arange(blk, device=DEV)        # [B, nbt, blk]
    t = slot - n_old[:, None, None]
    new = (t >= 0) & (t < n_new[:, None, None]) & inside[:, :, None]
    old = (t < 0) & inside[:, :, None]
    bi = torch.arange(B, device=DEV)
    xs = x.float()[bi[:, None, None], t.clamp(0, T - 1)]                   # [B, nbt, blk, H, d]
    fin = torch.where(new[..., None, None] & xs.isfinite(), xs.abs(), 0.0)
    amax = fin.amax((2, 4))                                                # [B, nbt, H]
    m, e = torch.frexp(amax)                                               # amax = m 2^e, m in [0.5, 1)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX)
    e_old = exps[bi[:, None], :, blocks].int() - 127                       # [B, nbt, H]
    has_old = old.any(2)[:, :, None]
    e_new = torch.where(has_old, torch.maximum(e, e_old), e)
    touched = new.any(2)[:, :, None] & inside[:, :, None]
    e_new = torch.where(touched, e_new, e_old)
    scale = _pow2(-e_new)[:, :, None, :, None]
    was = codes[bi[:, None, None], :, slot].view(torch.float8_e4m3fn)      # [B, nbt, blk, H, d]
    again = _e4m3(was.float() * _pow2(e_old - e_new)[:, :, None, :, None])
    keep = torch.where((old & touched)[..., None, None], again.view(torch.uint8), was.view(torch.uint8))
    got = torch.where(new[..., None, None], _e4m3(xs * scale).view(torch.uint8), keep)
    # a clamped block index repeats the last block: only real blocks are written
    at = inside.nonzero(as_tuple=True)
    codes.view(B, H, -1, blk, d)[at[0], :, blocks[at]] = got[at].transpose(1, 2)
    exps[at[0], :, blocks[at]] = (e_new[at] + 127).to(torch.uint8)


def _plain_append(s):
    c = s["c"]
    _plain_store(s["k"], s["n_old"], s["n_new"], s["kc"], s["k_exp"], c["block"])
    _plain_store(s["v"], s["n_old"], s["n_new"], s["vc"], s["v_exp"], c["block"])


def _values(codes, exps, blk):
    B, H, N, d = codes.shape
    x = codes.view(torch.float8_e4m3fn).float().view(B, H, N // blk, blk, d)
    return x.mul_(_pow2(exps.int() - 127)[..., None, None]).view(B, H, N, d)


def _plain_attend(s):
    c = s["c"]
    B, Q, H, d, N, blk = c["B"], c["Q"], c["n_kv"], c["d"], c["N"], c["block"]
    G = c["n_q"] // H
    q = s["q"].float().view(B, Q, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, Q * G, d)
    p = torch.matmul(q, _values(s["kc"], s["k_exp"], blk).transpose(2, 3)).mul_(d ** -0.5)
    vis = s["n_vis"].view(B, 1, Q, 1).expand(B, 1, Q, G).reshape(B, 1, Q * G, 1)
    p.masked_fill_(torch.arange(N, device=DEV) >= vis, -math.inf)
    top = p.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].view(1, H, 1, G).expand(B, H, Q, G).reshape(B, H, Q * G, 1)
        top = torch.maximum(top, sink)
    top = torch.where(top.isinf(), 0.0, top)
    p = p.sub_(top).exp_()
    den = p.sum(-1, keepdim=True)
    if s["sink"] is not None:
        den = den + torch.exp(sink - top)
    p = p.div_(torch.where(den > 0, den, 1.0))
    o = torch.matmul(p, _values(s["vc"], s["v_exp"], blk))
    s["out"].copy_(o.view(B, H, Q, G, d).permute(0, 2, 1, 3, 4).reshape(B * Q, H * G, d))
    if s["acc"] is not None:
        s["acc"].add_(p.sum(2).view(B, H, N // blk, blk).sum(-1))


def _plain_evict(s):
    c = s["c"]
    B, H, NB = s["acc"].shape
    keep, recent, blk = c["keep"], c["recent"], c["block"]
    i = torch.arange(NB, device=DEV)
    nb = ((s["n_tok"] + blk - 1) // blk).long()[:, None, None]            # blocks in use
    over = nb > keep
    cand = (i < nb - recent).expand(B, H, NB)
    order = torch.sort(s["acc"], dim=-1, descending=True, stable=True)[1]
    order = order.gather(-1, torch.sort((~cand).int().gather(-1, order), dim=-1, stable=True)[1])
    rank = torch.empty_like(order).scatter_(-1, order, i.expand(B, H, NB))
    stays = torch.where(over, (cand & (rank < keep - recent)) | ((i >= nb - recent) & (i < nb)), i < nb)
    # slots below keep - 1 whose block goes take the kept blocks from keep - 1 up in
    # ascending order; slot keep - 1 takes the last block
    hole = over & ~stays & (i < keep - 1)
    mover = over & stays & (i >= keep - 1) & (i != nb - 1)
    src = torch.where(i < nb, i, -1).expand(B, H, NB).clone()
    place = torch.full_like(src, NB)
    ids = torch.full((B, H, NB + 1), -1, device=DEV, dtype=src.dtype)
    ids.scatter_(-1, torch.where(mover, mover.cumsum(-1) - 1, place), i.expand(B, H, NB))
    src = torch.where(hole, ids.gather(-1, (hole.cumsum(-1) - 1).clamp(min=0)), src)
    src = torch.where(over & (i == keep - 1), nb - 1, src)
    src = torch.where(over & (i >= keep), -1, src)
    s["kept"].copy_(src[..., :keep] if NB >= keep else torch.nn.functional.pad(src, (0, keep - NB), value=-1))
    s["acc_out"].copy_(torch.where(src >= 0, s["acc"].gather(-1, src.clamp(min=0)), 0.0))
    moved = ((src != i) & (src >= 0)).nonzero(as_tuple=True)
    frm = (moved[0], moved[1], src[moved])
    kb, vb = (s[n].view(B, H, NB, blk * c["d"]) for n in ("kc", "vc"))
    for t in (kb, vb, s["k_exp"], s["v_exp"]):
        t[moved] = t[frm]
    s["n_tok_out"].copy_(torch.where(over[:, 0, 0], keep * blk - (nb[:, 0, 0] * blk - s["n_tok"]), s["n_tok"]))


# --------------------------------------------------------------------- run --
def _own(s):
    """The framework's calls, with the parameter structures a program keeps."""
    from long_context_sparse_09_b200 import binding as bd
    c = s["c"]
    if c["op"] == "norm_rope":
        if "rope" not in s:
            s["rope"] = bd.rope_params(c["d"], c["rope"], layout="half" if c["half"] else "interleaved",
                                       mscale=_mscale(c))
        bd.csa_qk_norm_rope(s["rope"], s["turns"], s["pos"], s["q"], s["k"], s["q_out"], s["k_out"],
                            q_gain=s["gq"], k_gain=s["gk"], eps=c["eps"])
        return
    if "p" not in s:
        s["p"] = bd.kv8_params(c.get("n_q", c["n_kv"]), c["n_kv"], c["d"], c["block"], c["N"], c["act"])
    kv = (s["kc"], s["k_exp"], s["vc"], s["v_exp"])
    if c["op"] == "append":
        bd.csa_kv8_append(s["p"], s["k"], s["v"], s["n_old"], *kv, n_new=s["n_new"])
    elif c["op"] == "evict":
        bd.csa_kv8_evict(s["p"], c["keep"], c["recent"], s["acc"], s["n_tok"], *kv, s["kept"],
                         s["acc_out"], s["n_tok_out"])
    else:
        bd.csa_kv8_attend(s["p"], s["q"], s["n_vis"], *kv, s["out"], sink=s["sink"], acc=s["acc"])


def run(s):
    op = s["c"]["op"]
    if own:
        _own(s)
    elif op == "norm_rope":
        return _plain_norm_rope(s)
    elif op == "append":
        _plain_append(s)
    elif op == "evict":
        _plain_evict(s)
    else:
        _plain_attend(s)
    if op == "norm_rope":
        return [s["q_out"], s["k_out"]]
    if op == "attend":
        return [s["out"]] + ([s["acc"]] if s["acc"] is not None else [])
    cache = [s["kc"].view(torch.float8_e4m3fn), s["vc"].view(torch.float8_e4m3fn), s["k_exp"], s["v_exp"]]
    return cache + ([s["kept"], s["acc_out"], s["n_tok_out"]] if op == "evict" else [])


# ------------------------------------------------------------------- exact --
def _exact_codes(y):
    """Doubles rounded to the E4M3 grid, ties to even: three fraction bits above
    2^-6, steps of 2^-9 below, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _exact_store(x, old, new, codes, exps, blk):
    val = codes.view(torch.float8_e4m3fn).double()
    e8 = exps.long() - 127
    for b in range(x.shape[0]):
        at, end = old[b], min(old[b] + new[b], codes.shape[2])
        while at < end:
            i = at // blk
            stop = min(end, (i + 1) * blk)
            xs = x[b, at - old[b]: stop - old[b]].double()                       # [n, H, d]
            top = xs.abs().amax((0, 2))
            e = torch.ceil(torch.log2(top / 448.0))
            e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)               # log2 off by an ulp
            e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e)
            e = torch.where(top > 0, e, E_MIN).clamp(E_MIN, E_MAX).long()
            if at % blk:
                e = torch.maximum(e, e8[b, :, i])
                f = torch.exp2((e8[b, :, i] - e).double())[:, None, None]
                val[b, :, i * blk: at] = _exact_codes(val[b, :, i * blk: at] * f)
            val[b, :, at: stop] = _exact_codes(xs.transpose(0, 1) * torch.exp2(-e.double())[:, None, None])
            e8[b, :, i] = e
            at = stop
    return val


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "norm_rope":
        got = []
        D, off = c["rope"], c["d"] - c["rope"]
        ang = 2.0 * math.pi * torch.remainder(s["pos"].double()[:, None] * s["turns"], 1.0)
        z = torch.polar(torch.full_like(ang, _mscale(c)), ang)[:, None, :]
        for x, gain in ((s["q"], s["gq"]), (s["k"], s["gk"])):
            x = x.double()
            x = x / torch.sqrt(torch.mean(x * x, -1, keepdim=True) + c["eps"]) * gain.double()
            r = x[..., off:].reshape(x.shape[:-1] + ((2, D // 2) if c["half"] else (D // 2, 2)))
            r = r.transpose(-1, -2) if c["half"] else r
            r = torch.view_as_real(torch.view_as_complex(r.contiguous()) * z)
            x[..., off:] = (r.transpose(-1, -2) if c["half"] else r).reshape(x.shape[:-1] + (D,))
            got.append(x)
        return got
    if c["op"] == "append":
        old, new = _lens(c), _news(c)
        return [_exact_store(s["k"], old, new, s["kc"], s["k_exp"], c["block"]),
                _exact_store(s["v"], old, new, s["vc"], s["v_exp"], c["block"]), None, None]
    if c["op"] == "evict":
        return None        # moves and whole numbers only
    B, Q, H, d, blk = c["B"], c["Q"], c["n_kv"], c["d"], c["block"]
    G, NB = c["n_q"] // H, c["N"] // blk
    out = torch.zeros(B * Q, c["n_q"], d, dtype=torch.float64, device=DEV)
    acc = s["acc"].double() if s["acc"] is not None else None
    for b in range(B):
        vis = s["n_vis"][b * Q: (b + 1) * Q].repeat_interleave(G)[:, None]
        n = int(vis.max())
        if n == 0:
            continue
        for h in range(H):
            K, V = (t[b, h].view(torch.float8_e4m3fn)[:n].double()
                    * torch.exp2(e[b, h].double() - 127.0).repeat_interleave(blk)[:n, None]
                    for t, e in ((s["kc"], s["k_exp"]), (s["vc"], s["v_exp"])))
            q = s["q"][b * Q: (b + 1) * Q, h * G: (h + 1) * G].double().reshape(Q * G, d)
            l = q @ K.T / math.sqrt(d)
            l = torch.where(torch.arange(n, device=DEV) < vis, l, -math.inf)
            if s["sink"] is not None:
                l = torch.cat([l, s["sink"][h * G: (h + 1) * G].double().repeat(Q)[:, None]], 1)
            p = torch.nan_to_num(torch.softmax(l, 1))[:, :n]
            out[b * Q: (b + 1) * Q, h * G: (h + 1) * G] = (p @ V).view(Q, G, d)
            if acc is not None:
                w = torch.nn.functional.pad(p.sum(0), (0, NB * blk - n))
                acc[b, h] += w.view(NB, blk).sum(1)
    return [out] + ([acc] if acc is not None else [])
