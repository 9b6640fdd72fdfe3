"""The 8-bit KV cache path against its fp64 oracle (oracle/kv8.py): norm and
rotation, append, attention with accumulated weights, eviction, and a run of
them together.

Tolerances.  U = 2^-24 is half a step of fp32 relative to the value, 2^-8 of
bf16, 2^-12 of fp16 (the type the attention's probabilities are rounded to).
* norm + rotation: the gain of an element carries the rounded sum of squares
  (at most 16 sequential adds and 5 of a tree, halved by the root: 11 U),
  root, divide and two products (4 U); the rotation the angle's rounding
  (half turns in fp32: pi U), sine and cosine (2 ulp: 4 U), mscale and two
  products and a sum (4 U): at most 32 U (|a| + |b|), then the output's
  rounding.
* attention: logits are sums of d products accumulated in fp32 (tensor cores
  may truncate: a full step 2 U each), with q held to 2^-22 at least; a logit
  is off by at most eps = (2 d + 16) U * load + 8 U * |logit range| where
  load = max scale sum |q||k|, so weights by 2 eps; p is rounded to fp16
  (2^-11 with the block's power of two, bf16 activations; in the tensor-core
  forms after a polynomial that is off by 2^-18.5) or to two fp16
  terms (2^-22, fp32 activations) and summed over n / 16 steps of truncating
  fp32.  The output is off by at most (2 eps + p rounding + (n / 8 + 16) U)
  times sum p |v|, then its own rounding.
* append and eviction: exact.
"""
import contextlib

import numpy as np
import pytest
import torch

from oracle import kv8
from long_context_sparse_09_b200 import binding as bd
from gpu_util import DEV

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": U, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _clean_status(cuda_ok):
    bd.device_status()
    yield
    torch.cuda.synchronize()
    assert bd.device_status() == 0


def np64(t):
    return t.detach().double().cpu().numpy()


def within(got, ref, tol, what):
    assert np.all(np.isfinite(got)), what
    bad = np.abs(got - ref) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst by " \
        f"{(np.abs(got - ref) / np.maximum(tol, 1e-300)).max():.3g} tolerances"


# ------------------------------------------------------- norm and rotation --
NORM = [
    # act, R, n_q, n_kv, d, rope_dims, rope_off, layout, scaling, norm, gain
    ("bf16", 1, 64, 8, 128, 128, 0, "half", "parts", True, True),
    ("bf16", 7, 5, 1, 64, 32, 32, "interleaved", "none", True, False),
    ("f32", 33, 3, 3, 96, 96, 0, "half", "linear", True, True),
    ("f32", 300, 4, 0, 512, 64, 448, "interleaved", "parts", True, True),
    ("bf16", 65, 9, 2, 256, 34, 5, "half", "none", True, True),
    ("bf16", 3, 2, 1, 8, 8, 0, "interleaved", "none", False, False),
    ("f32", 2, 17, 4, 40, 2, 38, "half", "none", False, False),
    ("bf16", 4, 3, 2, 128, 0, 0, "half", "none", True, True),
    ("bf16", 5, 2, 1, 264, 264, 0, "interleaved", "linear", True, True),
    # several tokens a CTA: 4, 8, and more where heads are few
    ("f32", 701, 5, 2, 128, 128, 0, "interleaved", "parts", True, True),
    ("bf16", 2501, 33, 2, 64, 32, 32, "half", "linear", True, True),
    ("bf16", 19001, 1, 1, 64, 64, 0, "half", "none", True, True),
    ("bf16", 9603, 4, 3, 96, 48, 8, "interleaved", "none", True, True),
    ("bf16", 2603, 2, 1, 256, 34, 5, "half", "none", True, False),
    ("f32", 2402, 1, 1, 512, 64, 448, "interleaved", "none", True, True),
    ("f32", 4801, 2, 0, 256, 256, 0, "half", "none", True, True),
]
SCALE = dict(factor=8.0, orig_len=4096.0)


def norm_rope_case(act, R, n_q, n_kv, d, D, off, layout, scaling, norm, gain, seed=0, wide=0):
    g = torch.Generator().manual_seed(seed + R * 31 + d)
    row = (n_q + n_kv) * d + wide
    x = (torch.randn(R, row, generator=g) * 2).to(DT[act]).to(DEV)
    q, k = x[:, :n_q * d].view(R, n_q, d), x[:, n_q * d:(n_q + n_kv) * d].view(R, n_kv, d)
    pos = torch.randint(-5, 1 << 20, (R,), generator=g, dtype=torch.int32)
    pos[0] = (1 << 31) - 1
    gains = [torch.randn(d, generator=g) if gain else None for _ in range(2)]
    mscale = 1.2 if scaling == "parts" else 1.0
    rope = bd.rope_params(d, D, off, layout, scaling=scaling, mscale=mscale, **SCALE)
    kw = SCALE if scaling != "none" else {}
    return rope, q, k, pos, gains, mscale, kv8.turns(D, scaling=scaling, **kw)


@pytest.mark.parametrize("case", NORM, ids=[f"{c[0]}-R{c[1]}-d{c[4]}-{c[5]}at{c[6]}-{c[7]}" for c in NORM])
@pytest.mark.parametrize("wide", [0, 64])
def test_norm_rope(case, wide):
    act, R, n_q, n_kv, d, D, off, layout, scaling, norm, gain = case
    rope, q, k, pos, gains, mscale, t = norm_rope_case(*case, wide=wide)
    turns = bd.csa_rope_freqs(rope)
    # pow to 2 ulp of fp64, a few more operations
    assert np.all(np.abs(np64(turns) - t) <= 16 * 2.0 ** -53 * t)
    q_ref, k_ref = np64(q), np64(k)
    q_out = torch.empty(R, n_q, d, dtype=q.dtype, device=DEV)
    k_out = torch.empty(R, n_kv, d, dtype=q.dtype, device=DEV) if n_kv else None
    dev = [None if x is None else x.to(DEV) for x in gains]
    for call in range(2):   # into new tensors, then in place
        o = (q_out, k_out) if call == 0 else (q, k if n_kv else None)
        bd.csa_qk_norm_rope(rope, turns, pos.to(DEV), q, k if n_kv else None, *o, q_gain=dev[0],
                            k_gain=dev[1], norm=norm)
        for got, x, gn, what in ((o[0], q_ref, gains[0], "q"), (o[1], k_ref, gains[1], "k")):
            if got is None:
                continue
            # turns may differ by 16 half steps of fp64: at 2^31 tokens that is 2^31 * t * 2^-49 turns
            drift = 2 * np.pi * 2.0 ** 31 * 2.0 ** -49 * (t.max() if len(t) else 0.0)
            ref, mag = kv8.norm_rope(x, pos.numpy(), t, off, layout, gn, norm=norm, mscale=mscale)
            within(np64(got), ref, HALF[act] * np.abs(ref) + (32 * U + drift) * mag, f"{what} call {call}")


def test_norm_rope_of_nothing_and_of_zeros():
    rope = bd.rope_params(64, 64)
    turns = bd.csa_rope_freqs(rope)
    e = torch.empty(0, 4, 64, device=DEV)
    bd.csa_qk_norm_rope(rope, turns, torch.empty(0, dtype=torch.int32, device=DEV), e, None, e, None)
    z = torch.zeros(3, 4, 64, device=DEV)
    out = torch.full_like(z, float("nan"))
    bd.csa_qk_norm_rope(rope, turns, torch.arange(3, dtype=torch.int32, device=DEV), z, None, out, None)
    assert torch.equal(out, z)


# ------------------------------------------------------------------ append --
APPEND = [
    # act, B, T, H, d, block, N, n_old, n_new (None: T)
    ("bf16", 1, 1, 1, 64, 16, 16, [0], None),
    ("bf16", 3, 1, 2, 128, 64, 256, [63, 64, 255], None),
    ("bf16", 2, 100, 3, 64, 32, 192, [5, 31], [100, 37]),
    ("f32", 4, 33, 2, 128, 16, 128, [0, 95, 17, 40], [33, 33, 0, 1]),
    ("f32", 1, 300, 1, 256, 128, 384, [77], None),
    ("bf16", 2, 129, 1, 256, 128, 384, [127, 255], None),
    ("f32", 1, 0, 2, 64, 16, 32, [3], None),
]


def random_cache(B, H, N, d, block, seed, lo=112, hi=126):
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 256, (2, B, H, N, d), generator=g, dtype=torch.uint8)
    c[(c & 0x7f) == 0x7f] = 0x11
    return c, torch.randint(lo, hi, (2, B, H, N // block), generator=g, dtype=torch.uint8)


@pytest.mark.parametrize("case", APPEND, ids=[f"{c[0]}-B{c[1]}-T{c[2]}-d{c[4]}-blk{c[5]}" for c in APPEND])
@pytest.mark.parametrize("spread", [False, True])
def test_append_is_exact(case, spread):
    act, B, T, H, d, block, N, n_old, n_new = case
    g = torch.Generator().manual_seed(T * 7 + d)
    x = torch.randn(2, B, T, H, d, generator=g) * torch.exp(3 * torch.randn(2, B, T, 1, 1, generator=g))
    if x.numel():   # values whose scaling meets zeros, subnormals, ends of the range
        flat = x.view(-1)
        special = [0.0, -0.0, 1e-40, 3e38, -3e38, float("inf"), float("-inf"), 448.0, 1.75]
        at = torch.randint(0, flat.numel(), (len(special),), generator=g)
        flat[at] = torch.tensor(special) if T > 2 else torch.tensor([0.0, 1.75, -0.0] * 3)
    x = x.to(DT[act])
    p = bd.kv8_params(H, H, d, block, N, act)
    codes, exps = random_cache(B, H, N, d, block, 5)
    dc, de = codes.to(DEV), exps.to(DEV)
    xd = x.to(DEV)
    if spread:   # tokens as rows of a wider tensor
        wide = torch.zeros(2, B, T, 2 * H, d, dtype=x.dtype, device=DEV)
        wide[:, :, :, :H] = xd
        xd = wide[:, :, :, :H]
    new = None if n_new is None else torch.tensor(n_new, dtype=torch.int32, device=DEV)
    bd.csa_kv8_append(p, xd[0], xd[1], torch.tensor(n_old, dtype=torch.int32, device=DEV), dc[0], de[0],
                      dc[1], de[1], n_new=new)
    assert bd.device_status() == 0
    for i in range(2):
        c, e = codes[i].numpy().copy(), exps[i].numpy().copy()
        kv8.append(x[i].double().numpy(), n_old, n_new or [T] * B, c, e, block)
        assert np.array_equal(de[i].cpu().numpy(), e), f"exponents of {'kv'[i]}"
        got = dc[i].cpu().numpy()
        assert np.array_equal(kv8._TAB[got], kv8._TAB[c]), f"codes of {'kv'[i]}"


def test_append_token_by_token_from_uninitialised_blocks():
    """Blocks start afresh: what the memory held before does not matter."""
    B, T, H, d, block, N = 2, 40, 2, 64, 16, 48
    g = torch.Generator().manual_seed(9)
    x = torch.randn(2, B, T, H, d, generator=g) * torch.exp2(torch.arange(T) / 4.0)[:, None, None]
    p = bd.kv8_params(H, H, d, block, N, "f32")
    dc = torch.full((2, B, H, N, d), 255, dtype=torch.uint8, device=DEV)
    de = torch.full((2, B, H, N // block), 255, dtype=torch.uint8, device=DEV)
    c, e = np.zeros((2, B, H, N, d), np.uint8), np.zeros((2, B, H, N // block), np.uint8)
    for t in range(T):
        xt = x[:, :, t:t + 1].to(DEV)
        bd.csa_kv8_append(p, xt[0], xt[1], torch.full((B,), t, dtype=torch.int32, device=DEV), dc[0], de[0],
                          dc[1], de[1])
        for i in range(2):
            kv8.append(x[i, :, t:t + 1].double().numpy(), [t] * B, [1] * B, c[i], e[i], block)
    nb = -(-T // block)
    assert np.array_equal(de.cpu().numpy()[..., :nb], e[..., :nb])
    assert np.array_equal(dc.cpu().numpy()[..., :T, :], c[..., :T, :])
    assert (dc[..., T:, :] == 255).all() and (de[..., nb:] == 255).all()


def test_append_reports_bad_lengths_and_nan():
    B, T, H, d, block, N = 4, 8, 1, 64, 16, 32
    p = bd.kv8_params(H, H, d, block, N, "f32")
    x = torch.randn(B, T, H, d, device=DEV)
    full = torch.full((B, H, N, d), 7, dtype=torch.uint8, device=DEV)
    kc, vc = full.clone(), full.clone()
    ke, ve = (torch.full((B, H, N // block), 120, dtype=torch.uint8, device=DEV) for _ in range(2))
    old = torch.tensor([-1, 33, 28, 0], dtype=torch.int32, device=DEV)
    new = torch.tensor([8, 8, 8, 9], dtype=torch.int32, device=DEV)
    bd.csa_kv8_append(p, x, x, old, kc, ke, vc, ve, n_new=new)
    assert bd.device_status() == bd.DEV_BAD_INDEX
    assert torch.equal(kc[:2], full[:2])            # skipped
    assert torch.equal(kc[2, :, :16], full[2, :, :16]) and not torch.equal(kc[2, :, 28:], full[2, :, 28:])
    assert torch.equal(kc[3, :, 8:], full[3, :, 8:])  # n_new above T: T tokens
    x[0, 3, 0, 5] = float("nan")
    bd.csa_kv8_append(p, x, x, torch.zeros_like(old), kc, ke, vc, ve)
    assert bd.device_status() == bd.DEV_NAN
    assert kc[0, 0, 3, 5] == 0 and ke[0, 0, 0] < 130


# ------------------------------------------------------------------ attend --
ATTEND = [
    # act, B, Q, n_q, n_kv, d, block, N, n_vis, sink, acc
    ("bf16", 1, 1, 1, 1, 64, 16, 16, [1], False, False),
    ("bf16", 2, 1, 8, 2, 128, 64, 192, [0, 65], True, True),
    ("f32", 2, 1, 6, 6, 64, 32, 96, [96, 33], False, True),
    ("bf16", 3, 1, 14, 2, 128, 16, 2048, [2048, 1, 1337], False, True),
    ("f32", 1, 3, 12, 3, 256, 128, 640, [538, 539, 540], True, False),
    ("bf16", 1, 5, 32, 1, 64, 32, 1024, [997, 998, 999, 1000, 1001], False, True),
    ("bf16", 2, 4, 16, 16, 256, 64, 320, [0, 1, 0, 320, 64, 63, 128, 7], True, True),
    ("bf16", 1, 70, 8, 2, 128, 64, 256, list(range(100, 170)), False, False),
    ("bf16", 2, 33, 6, 3, 64, 16, 128, list(range(-2, 31)) + list(range(96, 129)), True, True),
    ("f32", 1, 40, 4, 4, 128, 32, 160, list(range(1, 160, 4)), True, True),
    ("bf16", 1, 150, 8, 1, 128, 128, 512, list(range(0, 300, 2)), True, False),
    ("bf16", 1, 300, 2, 1, 64, 64, 384, list(range(1, 301)), False, True),
]


def attend_tol(act, d, n, ref, mag, load, scale_range):
    eps = (2 * d + 16) * U * load[..., None] + 8 * U * scale_range
    p_round = 2.0 ** -11 + 2.0 ** -18 if act == "bf16" else 2.0 ** -22
    return HALF[act] * np.abs(ref) + (2 * eps + p_round + (n / 8 + 16) * U) * mag


def attend_inputs(case, seed, garbage=True):
    act, B, Q, n_q, n_kv, d, block, N, n_vis, sink, acc = case
    g = torch.Generator().manual_seed(seed)
    codes, exps = random_cache(B, n_kv, N, d, block, seed, 115, 121)
    codes = (torch.randn(codes.shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    q = (torch.randn(B * Q, n_q, d, generator=g) * 2).to(DT[act])
    vis = torch.tensor(n_vis, dtype=torch.int32)
    clean = codes.clone()
    if garbage:   # NaN codes and wild exponents in slots that nothing sees
        for b in range(B):
            top = max(0, int(vis[b * Q:(b + 1) * Q].max()))
            codes[:, b, :, top:] = 0x7f
            exps[:, b, :, -(-top // block):] = 255
    z = torch.randn(n_q, generator=g) * 3 if sink else None
    w = torch.rand(B, n_kv, N // block, generator=g) if acc else None
    return clean, codes, exps, q, vis, z, w


def check_attend(case, seed, decay=1.0):
    act, B, Q, n_q, n_kv, d, block, N, n_vis, sink, acc = case
    clean, codes, exps, q, vis, z, w = attend_inputs(case, seed)
    p = bd.kv8_params(n_q, n_kv, d, block, N, act)
    dc, de = codes.to(DEV), exps.to(DEV)
    out = torch.full((B * Q, n_q, d), float("nan"), dtype=DT[act], device=DEV)
    dw = None if w is None else w.to(DEV)
    if decay == 0.0 and dw is not None:
        dw.fill_(float("nan"))
    # nothing in the workspace needs to be set: it starts as NaN
    ws = torch.full((bd.kv8_attend_workspace_bytes(p, B, Q, acc),), 255, dtype=torch.uint8, device=DEV)
    bd.csa_kv8_attend(p, q.to(DEV), vis.to(DEV), dc[0], de[0], dc[1], de[1], out,
                      sink=None if z is None else z.to(DEV), acc=dw, decay=decay, workspace=ws)
    exps_ref = np.where(exps.numpy() == 255, 127, exps.numpy())
    K, V = (kv8.values(clean[i].numpy(), exps_ref[i], block) for i in range(2))
    scale = d ** -0.5
    ref, wref, mag, load = kv8.attend(q.double().numpy(), n_vis, K, V, block, scale,
                                      None if z is None else z.double().numpy())
    rng = float(load.max(initial=0.0))
    within(np64(out), ref, attend_tol(act, d, N, ref, mag, load, rng) + 1e-30, "out")
    if dw is not None:
        # every weight by 2 eps and the sums over a block's slots and the rows
        eps = (2 * d + 16) * U * load.max(initial=0.0) + 8 * U * rng
        got = np64(dw)
        for b in range(B):
            top = -(-max(0, max(n_vis[b * Q:(b + 1) * Q])) // block)
            old = decay * w[b, :, :top].double().numpy() if decay else 0.0
            within(got[b, :, :top], old + wref[b, :, :top],
                   (2 * eps + (N / 8 + 2 * block + Q * n_q // n_kv + 24) * U) * wref[b, :, :top] + 2 * U * old + 1e-30, "acc")
            rest = got[b, :, top:]   # blocks no query sees: untouched
            assert np.isnan(rest).all() if decay == 0.0 else np.array_equal(rest, w[b, :, top:].double().numpy())
    return out, dw


IDS = [f"{c[0]}-B{c[1]}-Q{c[2]}-h{c[3]}of{c[4]}-d{c[5]}-blk{c[6]}" for c in ATTEND]


@pytest.mark.parametrize("case", ATTEND, ids=IDS)
def test_attend(case):
    check_attend(case, 11)


@pytest.mark.parametrize("decay", [0.0, 0.75])
def test_attend_decay(decay):
    check_attend(ATTEND[3], 12, decay)
    check_attend(ATTEND[8], 12, decay)


def test_attend_is_repeatable_bit_for_bit():
    case = ("bf16", 2, 1, 16, 2, 128, 64, 8192, [8000, 5000], True, True)
    a, wa = check_attend(case, 13)
    b, wb = check_attend(case, 13)
    assert torch.equal(a, b) and torch.equal(wa, wb)


@pytest.mark.parametrize("Q", [1, 2, 65, 2000])
def test_attend_extreme_values(Q):
    """Query magnitudes far from 1, block exponents far apart, logits that
    leave one slot, and a slot with a tiny value that takes all weight."""
    B, n_q, n_kv, d, block, N = 1, 4, 2, 64, 16, 64
    p = bd.kv8_params(n_q, n_kv, d, block, N, "bf16")
    codes, exps = random_cache(B, n_kv, N, d, block, 3, 118, 122)
    for qmag, kexp, vexp in ((1e-30, 127 + 90, 127 - 100), (1e30, 127 - 100, 127 + 90), (1.0, 120, 127)):
        e = exps.clone()
        e[0] = kexp - 4
        e[0, :, :, 1] = kexp
        e[1] = vexp
        e[1, :, :, 1] = vexp - 20
        q = (torch.randn(B * Q, n_q, d, generator=torch.Generator().manual_seed(4)) * qmag).to(torch.bfloat16)
        vis = [50] * Q
        K, V = (kv8.values(codes[i].numpy(), e[i].numpy(), block) for i in range(2))
        K[:, :, 50:] = V[:, :, 50:] = 0
        qs = q.double().numpy()
        scale = 2.0 / np.abs(np.einsum("rhd,hnd->rhn", qs, np.repeat(K[0], 2, 0))).std()
        out = torch.empty(B * Q, n_q, d, dtype=torch.bfloat16, device=DEV)
        dc, de = codes.to(DEV), e.to(DEV)
        bd.csa_kv8_attend(p, q.to(DEV), torch.tensor(vis, dtype=torch.int32, device=DEV), dc[0], de[0], dc[1],
                          de[1], out, scale=float(np.float32(scale)))
        ref, _, mag, load = kv8.attend(qs, vis, K, V, block, float(np.float32(scale)))
        rng = float(load.max())
        within(np64(out), ref, attend_tol("bf16", d, N, ref, mag, load, rng), f"q {qmag}")


@pytest.mark.parametrize("act,Q,rows", [("bf16", 3, 16), ("f32", 3, 16), ("bf16", 400, 128), ("f32", 700, 128), ("bf16", 700, 256)])
def test_attend_keeps_rows_apart(act, Q, rows):
    """A query of NaN or infinities leaves the others' results as they are."""
    B, n_q, n_kv, d, block, N = 1, 32, 4, 64, 16, 160
    p = bd.kv8_params(n_q, n_kv, d, block, N, act)
    case = (act, B, Q, n_q, n_kv, d, block, N, [N - 7] * Q, False, False)
    _, codes, exps, q, vis, _, _ = attend_inputs(case, 61)
    dc, de, qd, vd = codes.to(DEV), exps.to(DEV), q.to(DEV), vis.to(DEV)
    want = torch.empty_like(qd)
    with rows_of_a_cta(rows):
        bd.csa_kv8_attend(p, qd, vd, dc[0], de[0], dc[1], de[1], want)
    for bad in (float("nan"), float("inf")):
        got, qb = torch.empty_like(qd), qd.clone()
        qb[1, 5, 3] = bad
        bd.csa_kv8_attend(p, qb, vd, dc[0], de[0], dc[1], de[1], got)
        assert got[1, 5].isnan().all()
        got[1, 5] = want[1, 5]
        assert torch.equal(got, want)


@pytest.mark.parametrize("act,Q,d", [("bf16", 1, 128), ("bf16", 2300, 64), ("f32", 700, 128), ("bf16", 700, 256)])
def test_attend_in_two_graphs_and_on_two_streams(act, Q, d):
    """Two captured calls with a workspace each, replayed on streams of their own
    at the same time, with other lengths than at capture."""
    B, n_q, n_kv, block, N = 1, 32, 4, 32, 352
    p = bd.kv8_params(n_q, n_kv, d, block, N, act)
    runs = []
    for seed in (71, 72):
        case = (act, B, Q, n_q, n_kv, d, block, N, [N] * Q, False, True)
        _, codes, exps, q, vis, _, w = attend_inputs(case, seed)
        t = [x.to(DEV) for x in (codes, exps, q, vis, w)]
        t.append(torch.empty_like(t[2]))
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            bd.csa_kv8_attend(p, t[2], t[3], t[0][0], t[1][0], t[0][1], t[1][1], t[5], acc=t[4])
        runs.append((t, w.to(DEV), s, g))
    for t, w, s, g in runs:
        t[3].copy_(torch.arange(N - Q + 1, N + 1, dtype=torch.int32) if Q <= N else
                   torch.arange(Q, dtype=torch.int32) % (N + 1))
    torch.cuda.synchronize()
    for _ in range(3):
        for t, w, s, g in runs:
            with torch.cuda.stream(s):
                t[4].copy_(w)
                g.replay()
    torch.cuda.synchronize()
    for t, w, s, g in runs:
        out, acc = torch.empty_like(t[5]), w.clone()
        bd.csa_kv8_attend(p, t[2], t[3], t[0][0], t[1][0], t[0][1], t[1][1], out, acc=acc)
        assert torch.equal(out, t[5]) and torch.equal(acc, t[4])


@pytest.mark.parametrize("act,Q,rows", [("bf16", 3, 16), ("f32", 3, 16), ("bf16", 400, 128), ("f32", 700, 128), ("bf16", 700, 256)])
@pytest.mark.parametrize("kind", ["scale 0", "negative scale", "underflow"])
def test_attend_flat_and_turned_logits(act, Q, rows, kind):
    """Logits that are all 0, by their scale or because query times key is below
    any number, next to masked slots; and a scale below 0."""
    B, n_q, n_kv, d, block, N = 1, 32, 4, 64, 16, 160
    p = bd.kv8_params(n_q, n_kv, d, block, N, act)
    n_vis = [(7 * j) % (N + 1) for j in range(Q)]
    clean, codes, exps, q, vis, _, _ = attend_inputs((act, B, Q, n_q, n_kv, d, block, N, n_vis, False, False), 65)
    scale = {"scale 0": 0.0, "negative scale": -0.1, "underflow": 0.125}[kind]
    if kind == "underflow":
        q = (q.double() * 2.0 ** -110).to(DT[act])
        exps[0][exps[0] != 255] = 17 + 10
    out = torch.full_like(q, float("nan"), device=DEV)
    dc, de = codes.to(DEV), exps.to(DEV)
    with rows_of_a_cta(rows):
        bd.csa_kv8_attend(p, q.to(DEV), vis.to(DEV), dc[0], de[0], dc[1], de[1], out, scale=scale)
    e = np.where(exps.numpy() == 255, 127, exps.numpy())
    K, V = (kv8.values(clean[i].numpy(), e[i], block) for i in range(2))
    some = slice(0, Q, max(1, Q // 50))
    ref, _, mag, load = kv8.attend(q[some].double().numpy(), n_vis[some], K, V, block, scale)
    within(np64(out[some]), ref, attend_tol(act, d, N, ref, mag, load, load.max()) + 1e-30, kind)


def test_attend_clamps_and_reports_a_length_beyond_the_cache():
    case = ("bf16", 2, 1, 4, 2, 64, 16, 64, [70, 64], False, False)
    _, codes, exps, q, _, _, _ = attend_inputs(case, 1, garbage=False)
    p = bd.kv8_params(4, 2, 64, 16, 64, "bf16")
    dc, de, qd = codes.to(DEV), exps.to(DEV), q.to(DEV)
    outs = []
    for v in ([70, 64], [64, 64]):
        outs.append(torch.empty_like(qd))
        bd.csa_kv8_attend(p, qd, torch.tensor(v, dtype=torch.int32, device=DEV), dc[0], de[0], dc[1], de[1], outs[-1])
        assert bd.device_status() == (bd.DEV_BAD_INDEX if v[0] == 70 else 0)
    assert torch.equal(*outs)


# many query rows a KV head: lengths around tile and block ends, in any order
def spread_vis(B, Q, N, seed):
    g = np.random.default_rng(seed)
    v = g.integers(-3, N + 1, B * Q)
    v[g.integers(0, B * Q, 6)] = [0, 1, N, 127 % N, 128 % N, 129 % N]
    return v.tolist()


MANY = [
    # act, B, Q, n_q, n_kv, d, block, N, seed, sink, acc
    ("bf16", 1, 130, 1, 1, 64, 16, 16, 1, False, True),
    ("bf16", 2, 65, 4, 2, 128, 16, 144, 2, True, True),
    ("bf16", 1, 40, 28, 4, 128, 64, 1088, 3, False, True),
    ("bf16", 3, 33, 16, 1, 64, 32, 2976, 4, True, False),
    ("bf16", 1, 129, 3, 3, 64, 128, 1408, 5, True, True),
    ("bf16", 2, 200, 4, 2, 128, 32, 640, 6, False, True),
    ("f32", 1, 129, 3, 1, 64, 64, 704, 7, True, True),
    ("f32", 1, 70, 4, 2, 128, 16, 528, 8, False, True),
    ("bf16", 1, 45, 6, 2, 256, 32, 992, 9, True, True),
    ("bf16", 2, 300, 8, 2, 64, 64, 576, 10, False, True),
    ("bf16", 1, 520, 2, 1, 64, 16, 1040, 11, True, True),
]


@pytest.mark.parametrize("case", MANY, ids=[f"{c[0]}-B{c[1]}-Q{c[2]}-h{c[3]}of{c[4]}-d{c[5]}-blk{c[6]}-N{c[7]}" for c in MANY])
def test_attend_many_rows(case):
    act, B, Q, n_q, n_kv, d, block, N, seed, sink, acc = case
    check_attend((act, B, Q, n_q, n_kv, d, block, N, spread_vis(B, Q, N, seed), sink, acc), 20 + seed, 0.5)


@contextlib.contextmanager
def rows_of_a_cta(rows):
    """The attention calls inside go to the form whose CTAs own that many query
    rows (256 and 128: tcgen05)."""
    bd.profile_enable(True)
    try:
        bd.profile_collect()
        yield
        ran = {k for k, (_, n) in bd.profile_collect().items() if n and k.startswith("kv8_attend")}
    finally:
        bd.profile_enable(False)
    assert ran == {{16: "kv8_attend", 256: "kv8_attend_tc", 128: "kv8_attend_tc1"}[rows]}


WIDE = [
    # rows and KV heads enough for the tensor-core forms (rows of a CTA in front):
    # one tile, several, one line of units
    (256, "bf16", 2, 160, 64, 4, 64, 16, 48, 1, True, True),
    (256, "bf16", 1, 300, 64, 8, 128, 32, 160, 2, False, True),
    (256, "bf16", 2, 210, 48, 8, 128, 64, 704, 3, True, False),
    (128, "f32", 2, 70, 64, 4, 64, 32, 96, 6, True, True),
    (128, "f32", 1, 150, 64, 8, 128, 16, 272, 7, False, True),
    (128, "f32", 1, 300, 48, 6, 256, 64, 192, 8, True, False),
    (128, "f32", 1, 290, 14, 1, 128, 64, 4032, 9, True, True),
    (128, "bf16", 1, 150, 64, 8, 256, 16, 144, 10, True, True),
    (128, "bf16", 2, 300, 24, 4, 256, 128, 384, 11, False, True),
    (128, "bf16", 1, 290, 14, 1, 256, 32, 2016, 12, False, False),
    (128, "f32", 1, 290, 14, 1, 256, 16, 2000, 13, False, True),
    (128, "bf16", 2, 100, 64, 4, 64, 16, 272, 14, True, True),
    (128, "bf16", 4, 33, 64, 8, 128, 64, 704, 15, False, True),
    (128, "bf16", 1, 290, 14, 1, 128, 32, 2016, 16, True, False),
]


@pytest.mark.parametrize("case", WIDE, ids=[f"{c[0]}-{c[1]}-B{c[2]}-Q{c[3]}-h{c[4]}of{c[5]}-d{c[6]}-blk{c[7]}-N{c[8]}" for c in WIDE])
def test_attend_tensor_core_forms(case):
    rows, act, B, Q, n_q, n_kv, d, block, N, seed, sink, acc = case
    with rows_of_a_cta(rows):
        check_attend((act, B, Q, n_q, n_kv, d, block, N, spread_vis(B, Q, N, seed), sink, acc), 40 + seed, 0.5)


@pytest.mark.parametrize("d", [64, 128])
def test_attend_two_streams_on_one_line(d):
    """A prompt chunk whose row tiles several CTAs share; every 32nd query checked."""
    B, Q, n_q, n_kv, block, N = 1, 480, 14, 1, 32, 16384
    p = bd.kv8_params(n_q, n_kv, d, block, N, "bf16")
    n_vis = list(range(N - Q + 1, N + 1))
    n_vis[64] = 0
    clean, codes, exps, q, vis, z, _ = attend_inputs(("bf16", B, Q, n_q, n_kv, d, block, N, n_vis, True, False), 51)
    out = torch.full((Q, n_q, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = torch.full((bd.kv8_attend_workspace_bytes(p, B, Q, False),), 255, dtype=torch.uint8, device=DEV)
    dc, de = codes.to(DEV), exps.to(DEV)
    with rows_of_a_cta(256):
        bd.csa_kv8_attend(p, q.to(DEV), vis.to(DEV), dc[0], de[0], dc[1], de[1], out, sink=z.to(DEV), workspace=ws)
    some = slice(0, Q, 32)
    K, V = (kv8.values(clean[i].numpy(), exps[i].numpy(), block) for i in range(2))
    ref, _, mag, load = kv8.attend(q[some].double().numpy(), n_vis[some], K, V, block, d ** -0.5, z.double().numpy())
    within(np64(out[some]), ref, attend_tol("bf16", d, N, ref, mag, load, load.max()) + 1e-30, "out")
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("d,Q,n_q,n_kv,N", [(64, 296, 64, 8, 6144), (64, 64, 14, 1, 131072), (128, 300, 64, 8, 6112),
                                            (256, 64, 14, 1, 65536)])
def test_attend_long_fp32_sums(d, Q, n_q, n_kv, N):
    """fp32 prompts over so many slots that rows are summed up in parts of 2048,
    whole items and items that CTAs share.  A part is 2048 / 16 products of two
    terms, each truncated by 2 U at most; the parts add up rounded."""
    B, block = 1, 32
    p = bd.kv8_params(n_q, n_kv, d, block, N, "f32")
    n_vis = list(range(N - Q + 1, N + 1))
    n_vis[Q // 2] = 0
    clean, codes, exps, q, vis, _, _ = attend_inputs(("f32", B, Q, n_q, n_kv, d, block, N, n_vis, False, False), 91)
    some = [0, Q // 3, Q // 2, Q - 1]
    # one row's largest logits come late: its sum in memory is scaled down then
    q[Q - 1] = 0.5 * q[Q - 1] + torch.from_numpy(
        kv8.values(clean[0].numpy(), exps[0].numpy(), block)[0, :, N - 7].repeat(n_q // n_kv, 0)).float()
    out = torch.full((Q, n_q, d), float("nan"), device=DEV)
    dc, de = codes.to(DEV), exps.to(DEV)
    with rows_of_a_cta(128):
        bd.csa_kv8_attend(p, q.to(DEV), vis.to(DEV), dc[0], de[0], dc[1], de[1], out)
    K, V = (kv8.values(clean[i].numpy(), exps[i].numpy(), block) for i in range(2))
    ref, _, mag, load = kv8.attend(q[some].double().numpy(), [n_vis[i] for i in some], K, V, block, d ** -0.5)
    again = torch.full_like(out, float("nan"))
    bd.csa_kv8_attend(p, q.to(DEV), vis.to(DEV), dc[0], de[0], dc[1], de[1], again)
    assert torch.equal(again, out)
    eps = (2 * d + 16) * U * load[..., None] + 8 * U * load.max()
    within(np64(out[some]), ref, U * np.abs(ref) + (2 * eps + 2.0 ** -22 + (512 + N / 2048 + 16) * U) * mag + 1e-30, "out")
    # and the truncation's drift stays below 2^-18 of the output
    got = np64(out[some])
    assert abs((got * ref).sum() / (ref * ref).sum() - 1.0) < 2.0 ** -18


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_attend_one_tile_of_rows_a_cta(act):
    """More row tiles than one line of units holds: sequences without slots
    among them."""
    B, Q = 1030, 130
    vis = [(b * 37 + j) % 17 if b % 5 else 0 for b in range(B) for j in range(Q)]
    check_attend((act, B, Q, 1, 1, 64, 16, 16, vis, True, True), 31)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("Q,N", [(1, 20480), (80, 4096), (2000, 640)])
@pytest.mark.parametrize("kind", ["zeros first", "zeros between", "all zeros", "far apart"])
def test_attend_value_exponents_far_apart(act, Q, N, kind):
    """Blocks of zeros carry the least exponent; blocks of unlike size their
    own.  Logits do not depend on either, so neither may weights."""
    B, n_q, n_kv, d, block = 1, 4, 2, 64, 16
    p = bd.kv8_params(n_q, n_kv, d, block, N, act)
    g = torch.Generator().manual_seed(Q + N)
    codes = (torch.randn(2, B, n_kv, N, d, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    exps = torch.randint(115, 121, (2, B, n_kv, N // block), generator=g, dtype=torch.uint8)
    NB = N // block
    zero = {"zeros first": torch.arange(NB) < 3 * NB // 4, "zeros between": torch.arange(NB) % 3 == 1,
            "all zeros": torch.ones(NB, dtype=torch.bool), "far apart": torch.zeros(NB, dtype=torch.bool)}[kind]
    codes[1].view(B, n_kv, NB, block, d)[:, :, zero] = 0
    exps[1][:, :, zero] = 17
    if kind == "far apart":
        exps[1] = torch.tensor([17, 70, 127, 190, 246], dtype=torch.uint8)[torch.randint(0, 5, exps[1].shape, generator=g)]
    q = (torch.randn(B * Q, n_q, d, generator=g) * 2).to(DT[act])
    vis = torch.full((B * Q,), N - 5, dtype=torch.int32)
    acc = torch.zeros(B, n_kv, NB, device=DEV)
    out = torch.empty(B * Q, n_q, d, dtype=DT[act], device=DEV)
    dc, de = codes.to(DEV), exps.to(DEV)
    with rows_of_a_cta(16 if Q < 2000 else 128):
        bd.csa_kv8_attend(p, q.to(DEV), vis.to(DEV), dc[0], de[0], dc[1], de[1], out, acc=acc)
    K, V = (kv8.values(codes[i].numpy(), exps[i].numpy(), block) for i in range(2))
    ref, wref, mag, load = kv8.attend(q.double().numpy(), vis.tolist(), K, V, block, d ** -0.5)
    rng = load.max()
    tol = attend_tol(act, d, N, ref, mag, load, rng)
    # a term 2^7 2^(y - M) in fp16 is off by half its least step, 2^-25, at most where it is
    # subnormal: 2^-32 of the largest weight times 2^exponent, for each of N slots' codes up to 448
    # (few rows a KV head: 2^11 2^(y - M), so 2^-36)
    top = N * 2.0 ** (-36 if Q < 2000 else -32) * 448.0 * 2.0 ** (float(exps[1].max()) - 127.0) if kind == "far apart" else 0.0
    within(np64(out), ref, tol + top + 1e-36, "out")
    eps = (2 * d + 16) * U * rng + 8 * U * rng
    within(np64(acc), wref, (2 * eps + (N / 8 + 2 * block + Q * n_q // n_kv + 24) * U) * wref + 1e-30, "acc")


# ------------------------------------------------------------------- evict --
EVICT = [
    # B, H, d, block, N, n_tok, keep, recent
    (1, 1, 64, 16, 16, [16], 1, 1),
    (2, 2, 64, 16, 160, [153, 16], 1, 1),
    (3, 2, 128, 64, 640, [640, 321, 0], 4, 2),
    (2, 3, 64, 32, 3200, [3190, 1601], 50, 50),
    (1, 2, 256, 16, 1024, [1009], 63, 3),
    (2, 1, 64, 16, 40000, [39990, 20001], 700, 8),
    (1, 1, 64, 128, 8192, [8191], 64, 1),
    (3, 2, 128, 32, 1056, [1056, 800, 801], 25, 2),
    (2, 3, 64, 16, 640, [639, 512], 38, 30),
    (1, 4, 128, 64, 4096, [4090], 64, 1),
]


@pytest.mark.parametrize("case", EVICT, ids=[f"B{c[0]}-d{c[2]}-blk{c[3]}-N{c[4]}-keep{c[6]}" for c in EVICT])
@pytest.mark.parametrize("kind", ["random", "ties", "odd"])
@pytest.mark.parametrize("inplace", [False, True])
def test_evict_is_exact(case, kind, inplace):
    B, H, d, block, N, n_tok, keep, recent = case
    NB = N // block
    g = torch.Generator().manual_seed(NB + keep)
    acc = torch.rand(B, H, NB, generator=g) ** 3
    if kind == "ties":
        acc = torch.randint(0, 3, (B, H, NB), generator=g).float()
    elif kind == "odd":
        acc = torch.randn(B, H, NB, generator=g)
        acc[..., ::3] = float("nan")
        acc[..., 1::5] = float("-inf")
        acc[..., 2::7] = float("inf")
        acc[..., 4::9] = -0.0
    codes, exps = random_cache(B, H, N, d, block, NB)
    p = bd.kv8_params(H, H, d, block, N, "bf16")
    dc, de, da = codes.to(DEV), exps.to(DEV), acc.to(DEV)
    dn = torch.tensor(n_tok, dtype=torch.int32, device=DEV)
    ao, no = (da, dn) if inplace else (torch.full_like(da, 3.0), torch.full_like(dn, -5))
    kept = torch.full((B, H, keep), -7, dtype=torch.int32, device=DEV)
    bd.csa_kv8_evict(p, keep, recent, da, dn, dc[0], de[0], dc[1], de[1], kept, ao, no)
    ref_kept, ref_acc, ref_n = kv8.evict(acc.numpy(), n_tok, keep, recent, block)
    assert np.array_equal(kept.cpu().numpy(), ref_kept)
    assert np.array_equal(ao.cpu().numpy(), ref_acc, equal_nan=True)
    assert np.array_equal(no.cpu().numpy(), ref_n)
    for i in range(2):
        got = dc[i].cpu().view(B, H, NB, block * d)
        was = codes[i].view(B, H, NB, block * d)
        for b in range(B):
            for h in range(H):
                m = ref_kept[b, h][ref_kept[b, h] >= 0]
                assert torch.equal(got[b, h, :len(m)], was[b, h][torch.from_numpy(m).long()])
                assert torch.equal(got[b, h, keep:], was[b, h, keep:])
                assert np.array_equal(de[i, b, h, :len(m)].cpu().numpy(), exps[i, b, h].numpy()[m])
                assert torch.equal(de[i, b, h, keep:].cpu(), exps[i, b, h, keep:])




def test_evict_reports_a_bad_length():
    p = bd.kv8_params(1, 1, 64, 16, 64, "f32")
    codes, exps = random_cache(2, 1, 64, 64, 16, 1)
    dc, de = codes.to(DEV), exps.to(DEV)
    acc = torch.rand(2, 1, 4, device=DEV)
    a0 = acc.clone()
    n = torch.tensor([65, -1], dtype=torch.int32, device=DEV)
    kept = torch.empty(2, 1, 2, dtype=torch.int32, device=DEV)
    bd.csa_kv8_evict(p, 2, 1, acc, n, dc[0], de[0], dc[1], de[1], kept, acc, n)
    assert bd.device_status() == bd.DEV_BAD_INDEX
    assert (kept == -1).all() and torch.equal(acc, a0) and n.tolist() == [65, -1]
    assert torch.equal(dc.cpu(), codes)


# --------------------------------------------------------- offsets of 33 bits --
@pytest.mark.parametrize("act,Q,rows", [("bf16", 1, 16), ("bf16", 64, 256), ("f32", 48, 128)])
def test_a_cache_beyond_4_gb(act, Q, rows):
    """Append, attention and eviction in the last sequence of a cache of 5.4 GB of
    keys, the others empty."""
    B, n_q, n_kv, d, block, N, T = 5, 64, 8, 128, 64, 1 << 20, 200
    p = bd.kv8_params(n_q, n_kv, d, block, N, act)
    g = torch.Generator().manual_seed(81)
    kc, vc = (torch.empty(B, n_kv, N, d, dtype=torch.uint8, device=DEV) for _ in range(2))
    ke, ve = (torch.empty(B, n_kv, N // block, dtype=torch.uint8, device=DEV) for _ in range(2))
    x = torch.randn(2, B, T, n_kv, d, generator=g).to(DT[act])
    n = torch.tensor([0] * (B - 1) + [T], dtype=torch.int32, device=DEV)
    xd = x.to(DEV)
    bd.csa_kv8_append(p, xd[0], xd[1], torch.zeros_like(n), kc, ke, vc, ve, n_new=n)
    c, e = np.zeros((2, 1, n_kv, 256, d), np.uint8), np.zeros((2, 1, n_kv, 4), np.uint8)
    for i, (codes, exps) in enumerate(((kc, ke), (vc, ve))):
        kv8.append(x[i, B - 1:].double().numpy(), [0], [T], c[i], e[i], block)
        assert np.array_equal(codes[B - 1, :, :T].cpu().numpy(), c[i, 0, :, :T])
        assert np.array_equal(exps[B - 1, :, :4].cpu().numpy(), e[i, 0])
    q = (torch.randn(B * Q, n_q, d, generator=g) * 2).to(DT[act])
    vis = torch.cat([torch.zeros((B - 1) * Q, dtype=torch.int32), T - Q + 1 + torch.arange(Q, dtype=torch.int32)])
    out = torch.full((B * Q, n_q, d), float("nan"), dtype=DT[act], device=DEV)
    with rows_of_a_cta(rows):
        bd.csa_kv8_attend(p, q.to(DEV), vis.to(DEV), kc, ke, vc, ve, out)
    assert (out[:(B - 1) * Q] == 0).all()
    K, V = (kv8.values(c[i], e[i], block) for i in range(2))
    ref, _, mag, load = kv8.attend(q[(B - 1) * Q:].double().numpy(), vis[(B - 1) * Q:].tolist(), K, V, block, d ** -0.5)
    within(np64(out[(B - 1) * Q:]), ref, attend_tol(act, d, 256, ref, mag, load, load.max()) + 1e-30, "out")
    if Q > 1:
        return
    acc = torch.rand(B, n_kv, N // block, generator=g).to(DEV)
    want = kv8.evict(acc[B - 1:, :, :4].cpu().numpy(), [T], 2, 1, block)[0][0]
    kept = torch.empty(B, n_kv, 2, dtype=torch.int32, device=DEV)
    bd.csa_kv8_evict(p, 2, 1, acc, n, kc, ke, vc, ve, kept, acc, n)
    assert n.tolist() == [0] * (B - 1) + [T - 2 * block]
    assert np.array_equal(kept[B - 1].cpu().numpy(), want)
    for h in range(n_kv):
        blocks = c[0, 0, h].reshape(4, block, d)[want[h]].reshape(-1, d)[:T - 2 * block]
        assert np.array_equal(kc[B - 1, h, :T - 2 * block].cpu().numpy(), blocks)


# ------------------------------------------------------------ run together --
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_a_decode_run_with_eviction(act):
    """A prompt and a decode period: norm and rotation, append, attention with
    accumulated weights, eviction whenever a block over budget opens; every
    stage against the oracle on the stage's own inputs, the cache, lengths
    and weights carried along on the GPU alone."""
    B, n_q, n_kv, d, block, N, keep, recent, prompt, steps = 2, 4, 2, 64, 16, 96, 4, 2, 60, 40
    p = bd.kv8_params(n_q, n_kv, d, block, N, act)
    rope = bd.rope_params(d, 32, layout="half")
    turns = bd.csa_rope_freqs(rope)
    g = torch.Generator().manual_seed(21)
    kc, vc = (torch.zeros(B, n_kv, N, d, dtype=torch.uint8, device=DEV) for _ in range(2))
    ke, ve = (torch.zeros(B, n_kv, N // block, dtype=torch.uint8, device=DEV) for _ in range(2))
    acc = torch.zeros(B, n_kv, N // block, device=DEV)
    n_tok = torch.zeros(B, dtype=torch.int32, device=DEV)
    kept = torch.empty(B, n_kv, keep, dtype=torch.int32, device=DEV)
    c = [kc.cpu().numpy(), ke.cpu().numpy(), vc.cpu().numpy(), ve.cpu().numpy()]
    w, n, at = np.zeros(acc.shape), np.zeros(B, int), 0
    for step in range(steps):
        T = prompt if step == 0 else 1
        qkv = torch.randn(B * T, (n_q + 2 * n_kv) * d, generator=g).to(DT[act]).to(DEV)
        q, k = qkv[:, :n_q * d].view(-1, n_q, d), qkv[:, n_q * d:(n_q + n_kv) * d].view(-1, n_kv, d)
        v = qkv[:, (n_q + n_kv) * d:].view(B, T, n_kv, d)
        qo, ko = torch.empty(B * T, n_q, d, dtype=DT[act], device=DEV), torch.empty(B * T, n_kv, d, dtype=DT[act], device=DEV)
        pos = torch.arange(at, at + T, dtype=torch.int32, device=DEV).repeat(B)
        bd.csa_qk_norm_rope(rope, turns, pos, q, k, qo, ko)
        bd.csa_kv8_append(p, ko.view(B, T, n_kv, d), v, n_tok, kc, ke, vc, ve)
        vis = (n_tok[:, None] + 1 + torch.arange(T, dtype=torch.int32, device=DEV)).to(torch.int32).view(-1)
        n_tok += T
        out = torch.empty_like(qo)
        bd.csa_kv8_attend(p, qo, vis, kc, ke, vc, ve, out, acc=acc, decay=0.9)
        kv8.append(np64(ko).reshape(B, T, n_kv, d), n, [T] * B, c[0], c[1], block)
        kv8.append(np64(v), n, [T] * B, c[2], c[3], block)
        K, V = kv8.values(c[0], c[1], block), kv8.values(c[2], c[3], block)
        ref, wr, mag, load = kv8.attend(np64(qo), vis.tolist(), K, V, block, d ** -0.5)
        within(np64(out), ref, attend_tol(act, d, N, ref, mag, load, load.max()) + 1e-30, f"step {step}")
        n, at = n + T, at + T
        seen = np.arange(N // block) * block < n[:, None, None]
        w = np.where(seen, 0.9 * w, w) + wr
        # 40 steps of relative error 2 eps + sums, each fading by 0.9: below 10 of one step
        eps = 2 * (2 * d + 24) * U * load.max() + (N + T * n_q) * U
        within(np64(acc), w, 10 * eps * w + 1e-30, f"acc at step {step}")
        if n[0] > keep * block:
            bd.csa_kv8_evict(p, keep, recent, acc, n_tok, kc, ke, vc, ve, kept, acc, n_tok)
            kr, _, n = kv8.evict(w, n, keep, recent, block)
            assert np.array_equal(kept.cpu().numpy(), kr), f"step {step}"
            for b in range(B):
                for h in range(n_kv):
                    w[b, h, :keep], w[b, h, keep:] = w[b, h, kr[b, h]], 0.0
                    for codes, exps in ((c[0], c[1]), (c[2], c[3])):
                        blocks = codes[b, h].reshape(N // block, block, d)
                        blocks[:keep] = blocks[kr[b, h]]
                        exps[b, h, :keep] = exps[b, h][kr[b, h]]
            assert n_tok.tolist() == n.tolist()
    live = n[0]
    assert np.array_equal(kc.cpu().numpy()[:, :, :live], c[0][:, :, :live])
