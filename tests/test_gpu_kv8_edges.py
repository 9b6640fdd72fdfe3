"""Edges of the 8-bit KV cache path.  `attend64` is the attention in 64 bits on
the GPU, elementary torch operations, a KV head at a time; U = 2^-24 is half a
step of fp32.
"""
import numpy as np
import pytest
import torch

from oracle import kv8
from long_context_sparse_09_b200 import binding as bd
from gpu_util import DEV
from test_gpu_kv8 import DT, U, _clean_status, attend_tol, np64, random_cache, rows_of_a_cta, within  # noqa: F401

pytestmark = pytest.mark.gpu


def values64(codes, exps, block):
    """Stored values in doubles of codes [..][N][d] and exponent bytes."""
    e = torch.exp2(exps.double() - 127.0).repeat_interleave(block, -1)
    return codes.view(torch.float8_e4m3fn).double() * e[..., None]


def attend64(q, n_vis, codes, exps, block, scale, sink=None):
    """What oracle.kv8.attend returns, for tensors on the GPU: (out, weights by
    block, sum p |v|, largest scale sum |q||k| of each row)."""
    R, n_q, d = q.shape
    _, B, H, N, _ = codes.shape
    Q, G = R // B, n_q // H
    out, mag = (torch.zeros(R, n_q, d, dtype=torch.float64, device=DEV) for _ in range(2))
    load = torch.zeros(R, n_q, dtype=torch.float64, device=DEV)
    w = torch.zeros(B, H, N // block, dtype=torch.float64, device=DEV)
    step = max(1, (1 << 26) // (N * G))    # queries at a time
    for b in range(B):
        for h in range(H):
            K, V = (values64(codes[i, b, h], exps[i, b, h], block) for i in range(2))
            for j0 in range(0, Q, step):
                r = slice(b * Q + j0, b * Q + min(Q, j0 + step))
                at = (r, slice(h * G, (h + 1) * G))
                x = q[at].double()
                seen = torch.arange(N, device=DEV) < n_vis[r].clamp(0, N)[:, None, None]   # [n][1][N]
                l = torch.where(seen, scale * (x @ K.T), -torch.inf)
                load[at] = torch.where(seen, abs(scale) * (x.abs() @ K.abs().T), 0.0).amax(-1)
                top = l.amax(-1, keepdim=True)
                if sink is not None:
                    z = sink[h * G:(h + 1) * G].double()[:, None]
                    top = torch.maximum(top, z)
                top = torch.where(top.isinf(), 0.0, top)
                p = torch.exp(l - top)
                den = p.sum(-1, keepdim=True)
                if sink is not None:
                    den = den + torch.exp(z - top)
                p = torch.where(seen, p / den, 0.0)
                out[at], mag[at] = p @ V, p @ V.abs()
                w[b, h] += p.sum((0, 1)).view(N // block, block).sum(-1)
    return out.cpu().numpy(), w.cpu().numpy(), mag.cpu().numpy(), load.cpu().numpy()


def ordinary_codes(shape, g, std=60.0):
    return (torch.randn(shape, generator=g) * std).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


# ------------------------------------------------------------------- evict --
@pytest.mark.parametrize("NB,keep", [(3, 2), (40, 17), (40, 36), (1200, 300)])
def test_evict_ties_of_both_zeros(NB, keep):
    """0 and -0 are equal: of tied blocks the lower index stays."""
    block, d, recent = 16, 64, 1
    acc = torch.zeros(1, 2, NB)
    acc[..., ::2] = -0.0
    acc[0, 1] = -acc[0, 1]
    acc[..., 5::7] = 1.0
    acc[..., -1] = 1.0
    codes, exps = random_cache(1, 2, NB * block, d, block, NB)
    p = bd.kv8_params(2, 2, d, block, NB * block, "bf16")
    dc, de, da = codes.to(DEV), exps.to(DEV), acc.to(DEV)
    n = torch.tensor([NB * block], dtype=torch.int32, device=DEV)
    kept = torch.full((1, 2, keep), -7, dtype=torch.int32, device=DEV)
    acc_out, n_out = torch.empty_like(da), torch.empty_like(n)
    bd.csa_kv8_evict(p, keep, recent, da, n, dc[0], de[0], dc[1], de[1], kept, acc_out, n_out)
    ref, ref_acc, _ = kv8.evict(acc.numpy(), [NB * block], keep, recent, block)
    assert np.array_equal(kept.cpu().numpy(), ref)
    assert np.array_equal(acc_out.cpu().numpy(), ref_acc)
    for h in range(2):
        was = codes[0, 0, h].view(NB, block, d)[torch.from_numpy(ref[0, h]).long()]
        assert torch.equal(dc[0, 0, h].cpu().view(NB, block, d)[:keep], was)


# ------------------------------------------------------------------ append --
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_append_of_no_tokens_writes_nothing(act):
    """Sequences without new tokens keep every byte, exponents that the library
    would not write among them."""
    B, T, H, d, block, N = 4, 3, 2, 64, 16, 48
    p = bd.kv8_params(H, H, d, block, N, act)
    codes, exps = random_cache(B, H, N, d, block, 7)
    exps[:, :, :, 0], exps[:, :, :, 1] = 255, 3
    dc, de = codes.to(DEV), exps.to(DEV)
    x = torch.randn(2, B, T, H, d).to(DT[act]).to(DEV)
    old = torch.tensor([5, 17, 32, 48], dtype=torch.int32, device=DEV)
    bd.csa_kv8_append(p, x[0], x[1], old, dc[0], de[0], dc[1], de[1], n_new=torch.zeros_like(old))
    assert torch.equal(dc.cpu(), codes) and torch.equal(de.cpu(), exps)


# --------------------------------------------------------- warps partly in use --
@pytest.mark.parametrize("d,N", [(64, 6144), (128, 6112), (256, 4160)])
def test_attend_fp32_parts_with_a_warp_partly_in_use(d, N):
    """Whole items of more than 2048 slots (their rows are summed up in parts),
    the last warp of a tile with 24 rows of its 32."""
    Q, n_q, n_kv, block = 287, 64, 8, 32
    p = bd.kv8_params(n_q, n_kv, d, block, N, "f32")
    assert Q * n_q // n_kv % 32 == 24 and bd.kv8_attend_workspace_bytes(p, 1, Q) == 0   # no pieces: a CTA an item
    g = torch.Generator().manual_seed(d)
    codes = ordinary_codes((2, 1, n_kv, N, d), g).to(DEV)
    exps = torch.randint(115, 121, (2, 1, n_kv, N // block), generator=g, dtype=torch.uint8).to(DEV)
    q = (2 * torch.randn(Q, n_q, d, generator=g)).to(DEV)
    vis = torch.arange(N - Q + 1, N + 1, dtype=torch.int32, device=DEV)
    vis[100] = 0
    out = torch.full_like(q, float("nan"))
    with rows_of_a_cta(128):
        bd.csa_kv8_attend(p, q, vis, codes[0], exps[0], codes[1], exps[1], out)
    some = [0, 15, 16, 99, 100, 284, 285, 286]
    ref, _, mag, load = attend64(q[some].contiguous(), vis[some], codes, exps, block, d ** -0.5)
    # a part is 2048 / 16 products of two terms, each truncated by 2 U at most; the
    # parts add up rounded
    eps = (2 * d + 16) * U * load[..., None] + 8 * U * load.max()
    within(np64(out[some]), ref, U * np.abs(ref) + (2 * eps + 2.0 ** -22 + (512 + N / 2048 + 16) * U) * mag + 1e-30, "out")
    assert torch.isfinite(out).all()


# ------------------------------------------------------ sums over long caches --
def drift_of(got, ref):
    return (got * ref).sum() / (ref * ref).sum() - 1.0


@pytest.mark.parametrize("d,H", [(64, 4), (128, 4), (256, 4)])
def test_attend_fp32_decode_sums_do_not_drift(d, H):
    """One query over 128K slots that one CTA walks, values of one sign: an
    accumulator that cuts off what it adds would lose 4e-5 of them.  The rounded
    sums stay within 2^-18, the bound that prompts have."""
    B, N, block = 37, 131072 if d < 256 else 65536, 64
    p = bd.kv8_params(H, H, d, block, N, "f32")
    g = torch.Generator(device=DEV).manual_seed(5)
    codes = torch.randint(0x30, 0x50, (2, B, H, N, d), generator=g, device=DEV, dtype=torch.uint8)
    exps = torch.full((2, B, H, N // block), 125, dtype=torch.uint8, device=DEV)
    q = 0.05 * torch.randn(B, H, d, generator=g, device=DEV)
    vis = torch.full((B,), N - 9, dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    bd.csa_kv8_attend(p, q, vis, codes[0], exps[0], codes[1], exps[1], out)
    some = [0, 17, 36]
    ref, _, mag, load = attend64(q[some], vis[some], codes[:, some], exps[:, some], block, d ** -0.5)
    got = np64(out[some])
    assert abs(drift_of(got, ref)) < 2.0 ** -18, drift_of(got, ref)
    eps = (2 * d + 16) * U * load[..., None] + 8 * U * load.max()
    # a warp's sums: N / 12 / 16 rounded steps at most (fewer warps: N / 6 / 16)
    within(got, ref, U * np.abs(ref) + (2 * eps + 2.0 ** -22 + (N / (96 if d == 256 else 192) + 16) * U) * mag, "out")


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_fp32_decode_parts_under_a_rising_reference(d, weights):
    """Logits that rise with the slot: the sums of earlier parts count, scaled
    down.  Rows of one CTA that see all slots, less than a part, and none."""
    B, Q, H, n_q, block = 37, 2, 4, 8, 64
    N = {64: 49152, 128: 36864, 256: 18432}[d]
    p = bd.kv8_params(n_q, H, d, block, N, "f32")
    g = torch.Generator(device=DEV).manual_seed(6)
    codes = torch.randint(0x30, 0x50, (2, B, H, N, d), generator=g, device=DEV, dtype=torch.uint8)
    ramp = torch.linspace(-440.0, 440.0, N, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[0, ..., 0] = ramp
    exps = torch.full((2, B, H, N // block), 125, dtype=torch.uint8, device=DEV)
    q = 0.02 * torch.randn(B * Q, n_q, d, generator=g, device=DEV)
    q[..., 0] = 8.0 * d ** 0.5 / 110.0    # logits from -8 to 8
    vis = torch.full((B, Q), N - 9, dtype=torch.int32, device=DEV)
    vis[::3, 1], vis[1::3, 0] = 1500, 0
    vis = vis.view(-1).contiguous()
    out = torch.empty_like(q)
    acc = torch.zeros(B, H, N // block, device=DEV) if weights else None
    with rows_of_a_cta(16):
        bd.csa_kv8_attend(p, q, vis, codes[0], exps[0], codes[1], exps[1], out, acc=acc)
    some = torch.tensor([0, 1, 2, 18, 36], device=DEV)
    rows = (some[:, None] * Q + torch.arange(Q, device=DEV)).view(-1)
    ref, w, mag, load = attend64(q[rows], vis[rows], codes[:, some].contiguous(), exps[:, some].contiguous(), block, d ** -0.5)
    eps = (2 * d + 16) * U * load[..., None] + 8 * U * load.max()
    within(np64(out[rows]), ref, U * np.abs(ref) + (2 * eps + 2.0 ** -22 + (N / 96 + 16) * U) * mag, "out")
    if weights:
        eps = (2 * d + 16) * U * load.max() + 8 * U * load.max()
        within(np64(acc[some]), w, (2 * eps + (N / 8 + 2 * block + 4 + 24) * U) * w + 1e-30, "acc")


# ------------------------------------------------------- ends of fp32's range --
FORMS = [  # act, B, Q, n_q, n_kv, d, N, rows of a CTA
    ("bf16", 1, 3, 32, 4, 64, 160, 16), ("f32", 1, 3, 32, 4, 64, 160, 16), ("bf16", 1, 400, 32, 4, 64, 160, 128),
    ("f32", 1, 700, 32, 4, 64, 160, 128), ("bf16", 1, 700, 32, 4, 64, 160, 256),
    ("f32", 1, 1, 4, 2, 64, 20480, 16), ("f32", 1, 290, 14, 1, 128, 4032, 128)]
FORM_IDS = [f"{c[0]}-Q{c[2]}-d{c[5]}-N{c[6]}-rows{c[7]}" for c in FORMS]


def run_form(case, codes, exps, q, vis, block, scale, sink=None, acc=None, decay=1.0):
    act, B, Q, n_q, n_kv, d, N, rows = case
    p = bd.kv8_params(n_q, n_kv, d, block, N, act)
    out = torch.full((B * Q, n_q, d), float("nan"), dtype=DT[act], device=DEV)
    ws = torch.full((bd.kv8_attend_workspace_bytes(p, B, Q, acc is not None),), 255, dtype=torch.uint8, device=DEV)
    with rows_of_a_cta(rows):
        bd.csa_kv8_attend(p, q, vis, codes[0], exps[0], codes[1], exps[1], out, sink=sink, scale=scale, acc=acc,
                          decay=decay, workspace=ws)
    return out


@pytest.mark.parametrize("case", FORMS, ids=FORM_IDS)
def test_attend_tiny_queries_over_large_keys(case):
    """Queries of 1e-35 and keys of 1e34: logits of a usual size."""
    act, B, Q, n_q, n_kv, d, N, rows = case
    g = torch.Generator().manual_seed(3)
    block = 32
    codes = ordinary_codes((2, B, n_kv, N, d), g).to(DEV)
    exps = torch.randint(120, 124, (2, B, n_kv, N // block), generator=g, dtype=torch.uint8).to(DEV)
    exps[0] += 112
    q = (torch.randn(B * Q, n_q, d, generator=g) * 1e-35).to(DT[act]).to(DEV)
    vis = torch.full((B * Q,), N - 7, dtype=torch.int32, device=DEV)
    out = run_form(case, codes, exps, q, vis, block, d ** -0.5)
    ref, _, mag, load = attend64(q, vis, codes, exps, block, d ** -0.5)
    assert 1.0 < load.max() < 100.0
    within(np64(out), ref, attend_tol(act, d, N, ref, mag, load, load.max()), "out")


@pytest.mark.parametrize("case", FORMS, ids=FORM_IDS)
def test_attend_tiny_values_under_a_large_sink(case):
    """Values of 2^-100 and a sink that takes all but 2^-30: outputs are still
    normal numbers, and as accurate as any."""
    act, B, Q, n_q, n_kv, d, N, rows = case
    g = torch.Generator().manual_seed(4)
    block = 32
    codes = ordinary_codes((2, B, n_kv, N, d), g)
    codes[1] &= 0x7f
    codes = codes.to(DEV)
    exps = torch.full((2, B, n_kv, N // block), 121, dtype=torch.uint8, device=DEV)
    exps[1] = 27
    q = (torch.randn(B * Q, n_q, d, generator=g) * 0.1).to(DT[act]).to(DEV)
    vis = torch.full((B * Q,), N - 7, dtype=torch.int32, device=DEV)
    sink = torch.full((n_q,), 30.3 * np.log(2.0) + np.log(N), device=DEV)
    out = run_form(case, codes, exps, q, vis, block, d ** -0.5, sink=sink)
    ref, _, mag, load = attend64(q, vis, codes, exps, block, d ** -0.5, sink)
    # the reference of y = x - 100 rounds by 2^-18 of a power of two; sink and logits of 32
    tol = attend_tol(act, d, N if N > 1000 else 0, ref, mag, load, load.max() + 32.0) + 2.0 ** -18 * mag
    within(np64(out), ref, tol, "out")


# --------------------------------------- weights of calls that run as several --
SHARED = [
    # act, B, Q, n_q, n_kv, d, block, N: queries of one sequence in turn (two tensor-core
    # calls; three on mma.sync), sequences in turn
    ("bf16", 1, 4200, 8, 1, 64, 16, 65536),
    ("f32", 1, 70, 64, 64, 64, 16, 1 << 20),
    ("bf16", 5, 500, 64, 8, 128, 16, 16384),
]


@pytest.mark.parametrize("decay", [1.0, 0.5, 0.0])
@pytest.mark.parametrize("case", SHARED, ids=[f"{c[0]}-B{c[1]}-Q{c[2]}-N{c[7]}" for c in SHARED])
def test_attend_weights_in_several_calls(case, decay):
    """Each query sees more than the one before, so later calls see blocks that
    earlier ones do not; the last blocks nobody sees."""
    act, B, Q, n_q, n_kv, d, block, N = case
    p = bd.kv8_params(n_q, n_kv, d, block, N, act)
    assert B * Q * n_q * (N // 16) * 4 > 512 << 20
    g = torch.Generator(device=DEV).manual_seed(8)
    codes = torch.randint(0, 0x58, (2, B, n_kv, N, d), generator=g, device=DEV, dtype=torch.uint8)
    codes[1] += torch.randint(0, 2, codes[1].shape, generator=g, device=DEV, dtype=torch.uint8) * 0x80
    exps = torch.full((2, B, n_kv, N // block), 121, dtype=torch.uint8, device=DEV)
    q = (0.2 * torch.randn(B * Q, n_q, d, generator=g, device=DEV)).to(DT[act])
    n_vis = (torch.linspace(-3, N - 4 * block - 5, Q, device=DEV).int() + 3 * torch.arange(B, device=DEV).int()[:, None])
    n_vis = n_vis.to(torch.int32).view(-1).contiguous()
    acc = torch.rand(B, n_kv, N // block, generator=g, device=DEV)
    was = acc.double().cpu().numpy()
    if decay == 0.0:
        acc.fill_(float("nan"))
    ws = torch.full((bd.kv8_attend_workspace_bytes(p, B, Q, True),), 255, dtype=torch.uint8, device=DEV)
    out = torch.full((B * Q, n_q, d), float("nan"), dtype=DT[act], device=DEV)
    bd.csa_kv8_attend(p, q, n_vis, codes[0], exps[0], codes[1], exps[1], out, acc=acc, decay=decay, workspace=ws)
    ref, w, mag, load = attend64(q, n_vis, codes, exps, block, d ** -0.5)
    within(np64(out), ref, attend_tol(act, d, N, ref, mag, load, load.max()) + 1e-30, "out")
    eps = (2 * d + 24) * U * load.max()
    for b in range(B):
        top = -(-int(n_vis[(b + 1) * Q - 1]) // block)
        old = decay * was[b, :, :top] if decay else 0.0
        # (one rounding more of the old weight, one for each call)
        within(np64(acc[b, :, :top]), old + w[b, :, :top],
               (2 * eps + (N / 8 + 2 * block + Q * n_q // n_kv + 24) * U) * w[b, :, :top] + 6 * U * old + 1e-30, "acc")
        rest = np64(acc[b, :, top:])
        assert np.isnan(rest).all() if decay == 0.0 else np.array_equal(rest, was[b, :, top:])


# ------------------------------------------------------- a stream of their own --
def test_calls_on_another_stream_take_no_memory_in_use():
    """Memory that was freed on the current stream may still be written there:
    what a call on another stream allocates must not be that memory."""
    s = torch.cuda.Stream()
    rope = bd.rope_params(128, 64)
    want = bd.csa_rope_freqs(rope)
    p = bd.kv8_params(8, 2, 64, 16, 20480, "bf16")
    need = bd.kv8_attend_workspace_bytes(p, 1, 1)
    codes, exps = random_cache(1, 2, 20480, 64, 16, 3)
    codes, exps = codes.to(DEV), exps.to(DEV)
    q = torch.randn(1, 8, 64, device=DEV).to(torch.bfloat16)
    vis = torch.tensor([20001], dtype=torch.int32, device=DEV)
    ref, out = torch.empty_like(q), torch.empty_like(q)
    bd.csa_kv8_attend(p, q, vis, codes[0], exps[0], codes[1], exps[1], ref)
    torch.cuda.synchronize()
    freed = torch.empty(32, dtype=torch.float64, device=DEV), torch.empty(need, dtype=torch.uint8, device=DEV)
    at = [t.data_ptr() for t in freed]
    torch.cuda._sleep(200_000_000)   # a tenth of a second
    for t in freed:
        t.fill_(255)
    del freed, t
    taken = []
    empty = torch.empty

    def watched(*args, **kw):
        t = empty(*args, **kw)
        taken.append(t.data_ptr())
        return t
    torch.empty = watched
    try:
        got = bd.csa_rope_freqs(rope, stream=s)
        bd.csa_kv8_attend(p, q, vis, codes[0], exps[0], codes[1], exps[1], out, stream=s)
    finally:
        torch.empty = empty
    assert len(taken) == 2 and not set(taken) & set(at)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(out, ref)


# ---------------------------------------------- value exponents far apart, by form --
FAR = [  # act, B, Q, n_q, n_kv, d, block, N, rows of a CTA
    ("bf16", 2, 210, 48, 8, 64, 16, 1296, 256), ("bf16", 1, 300, 64, 8, 64, 64, 1280, 256),
    ("bf16", 1, 300, 64, 8, 128, 16, 1296, 256), ("bf16", 2, 210, 48, 8, 128, 32, 1312, 256),
    ("bf16", 1, 480, 14, 1, 128, 32, 16384, 256),
    ("bf16", 1, 290, 14, 1, 128, 32, 2016, 128), ("bf16", 1, 150, 64, 8, 256, 16, 1296, 128),
    ("f32", 1, 150, 64, 8, 128, 16, 1296, 128), ("f32", 1, 300, 48, 6, 256, 64, 1280, 128)]
KINDS = ["zeros first", "zeros between", "far apart", "far from 200", "far from 700", "far from 1100"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", FAR, ids=[f"{c[0]}-d{c[5]}-blk{c[6]}-N{c[7]}-rows{c[8]}" for c in FAR])
def test_attend_value_exponents_far_apart_by_form(case, kind):
    """Logits do not depend on the values' exponents, so neither may weights; the
    first block out of the ordinary lies in any tile of a group of four, or in a
    later group."""
    act, B, Q, n_q, n_kv, d, block, N, rows = case
    g = torch.Generator().manual_seed(N + d)
    codes = ordinary_codes((2, B, n_kv, N, d), g)
    exps = torch.randint(115, 121, (2, B, n_kv, N // block), generator=g, dtype=torch.uint8)
    i = torch.arange(N // block)
    if kind.startswith("zeros"):
        zero = i < 3 * len(i) // 4 if kind == "zeros first" else i % 3 == 1
        codes[1].view(B, n_kv, -1, block, d)[:, :, zero] = 0
        exps[1][:, :, zero] = 17
    else:
        far = i * block >= (0 if kind == "far apart" else int(kind.split()[-1]) * N // 1280)
        wild = torch.tensor([17, 70, 127, 190, 246], dtype=torch.uint8)
        exps[1][:, :, far] = wild[torch.randint(0, 5, (B, n_kv, int(far.sum())), generator=g)]
    q = (2 * torch.randn(B * Q, n_q, d, generator=g)).to(DT[act]).to(DEV)
    vis = torch.from_numpy(np.random.default_rng(N).integers(N // 2, N + 1, B * Q).astype(np.int32))
    vis[5], vis[6], vis[7] = 0, 1, N // 3
    codes, exps, vis = codes.to(DEV), exps.to(DEV), vis.to(DEV)
    acc = torch.zeros(B, n_kv, N // block, device=DEV)
    out = run_form((act, B, Q, n_q, n_kv, d, N, rows), codes, exps, q, vis, block, d ** -0.5, acc=acc)
    ref, w, mag, load = attend64(q, vis, codes, exps, block, d ** -0.5)
    rng = load.max()
    # a term 2^7 2^(y - M) in fp16 is off by half its least step, 2^-25, at most where it is
    # subnormal: 2^-32 of the largest weight times 2^exponent, for each of N slots' codes up to 448
    top = 0.0 if kind.startswith("zeros") else N * 2.0 ** -32 * 448.0 * 2.0 ** (float(exps[1].max()) - 127.0)
    within(np64(out), ref, attend_tol(act, d, N, ref, mag, load, rng) + top + 1e-36, "out")
    eps = (2 * d + 24) * U * rng
    within(np64(acc), w, (2 * eps + (N / 8 + 2 * block + Q * n_q // n_kv + 24) * U) * w + 1e-30, "acc")


# ------------------------------------------- sums in parts whose reference leaps --
LEAP = [  # Q, n_q, n_kv, d, N, leaps at: whole items, and items that CTAs share
    (287, 64, 8, 64, 12288, (5000, 9000)), (287, 64, 8, 128, 12288, (4500, 9900)),
    (287, 64, 8, 256, 12288, (5300, 8300)), (64, 14, 1, 64, 131072, (60000, 100000)),
    (64, 14, 1, 128, 131072, (30000, 34000))]


@pytest.mark.parametrize("case", LEAP, ids=[f"d{c[3]}-N{c[4]}" for c in LEAP])
def test_attend_fp32_parts_when_the_reference_leaps(case):
    """Prompts of fp32 activations keep a row's sum of parts of 2048 slots in memory
    under the reference it began with; a rise beyond 2^60 scales that sum.  Every third
    query meets two such rises, one in a later part and one after that: the slots
    that cause them have no value in a third of the dims and only the first has
    one in another third, so that what was scaled down once and twice can be read
    off."""
    Q, n_q, n_kv, d, N, leaps = case
    block, tile = 32, 64 if d == 256 else 128
    p = bd.kv8_params(n_q, n_kv, d, block, N, "f32")
    g = torch.Generator().manual_seed(d + N)
    codes = torch.randint(0x30, 0x50, (2, 1, n_kv, N, d), generator=g, dtype=torch.uint8)
    codes[0] += torch.randint(0, 2, codes[0].shape, generator=g, dtype=torch.uint8) * 0x80
    level = torch.zeros(N)                       # logits of the leaping queries, in powers of two
    level[leaps[0] // tile * tile:] = -32.0      # what follows does not count
    level[leaps[0]], level[leaps[1]] = 64.0, 128.0
    codes[0, 0, :, :, 0] = level.to(torch.float8_e4m3fn).view(torch.uint8)
    codes[1, 0, :, leaps[0], 0::3] = 0
    codes[1, 0, :, leaps[1], 0::3] = 0
    codes[1, 0, :, leaps[1], 1::3] = 0
    exps = torch.full((2, 1, n_kv, N // block), 127, dtype=torch.uint8)
    exps[1] += 20
    q = 0.1 * torch.randn(Q, n_q, d, generator=g)
    q[..., 0] = 0.0
    q[::3, :, 0] = 1.1 * np.log(2.0) * d ** 0.5
    vis = torch.full((Q,), N - 3, dtype=torch.int32)
    vis[1] = leaps[0] + 40
    codes, exps, q, vis = codes.to(DEV), exps.to(DEV), q.to(DEV), vis.to(DEV)
    # the rises, from the logits in 64 bits
    K = values64(codes[0, 0, 0], exps[0, 0, 0], block)
    y = (q[0, :n_q // n_kv].double() @ K.T) * d ** -0.5 / np.log(2.0)
    steps = [y[:, :n].amax(-1) for n in (2048, leaps[0], leaps[0] + 1, leaps[1], leaps[1] + 1)]
    assert (steps[1] - steps[0]).max() < 8 and (steps[2] - steps[1]).min() > 60
    assert (steps[3] - steps[2]).max() == 0 and (steps[4] - steps[3]).min() > 60
    out = torch.full_like(q, float("nan"))
    with rows_of_a_cta(128):
        bd.csa_kv8_attend(p, q, vis, codes[0], exps[0], codes[1], exps[1], out)
    some = [0, 1, 2, 3, 30, Q // 3 * 3 - 3, Q - 1]
    ref, _, mag, load = attend64(q[some].contiguous(), vis[some], codes, exps, block, d ** -0.5)
    eps = (2 * d + 16) * U * load[..., None] + 8 * U * load.max()
    tol = U * np.abs(ref) + (2 * eps + 2.0 ** -22 + (512 + N / 2048 + 16) * U) * mag
    if Q == 64:   # pieces that lie more than 2^126 below the largest one are joined with a
        # factor of 0 (fp32 has no normal number there): N weights below 2^-126 of values
        # up to 448 2^20
        tol = tol + N * 2.0 ** -126 * 448 * 2.0 ** 20
    within(np64(out[some]), ref, tol, "out")
    assert torch.isfinite(out).all()


# ------------------------------------------------ bf16 sums over long caches --
@pytest.mark.parametrize("B,Q,n_q,n_kv,N,rows", [(37, 1, 4, 4, 1 << 18, 16), (37, 1, 4, 4, 1 << 20, 16),
                                                 (1, 592, 64, 4, 1 << 20, 256)])
def test_attend_bf16_sums_drift_less_than_their_rounding(B, Q, n_q, n_kv, N, rows):
    """What the tensor cores cut off an accumulator of values of one sign, one CTA an
    item (0.8% over 1M slots without parts), stays below a quarter of bf16's half
    step, 2^-10."""
    d, block = 64, 64
    g = torch.Generator(device=DEV).manual_seed(9)
    codes = torch.randint(0x30, 0x50, (2, B, n_kv, N, d), generator=g, device=DEV, dtype=torch.uint8)
    exps = torch.full((2, B, n_kv, N // block), 125, dtype=torch.uint8, device=DEV)
    q = (0.05 * torch.randn(B * Q, n_q, d, generator=g, device=DEV)).to(torch.bfloat16)
    vis = torch.full((B * Q,), N - 9, dtype=torch.int32, device=DEV)
    out = run_form(("bf16", B, Q, n_q, n_kv, d, N, rows), codes, exps, q, vis, block, d ** -0.5)
    some = [0, B * Q // 2, B * Q - 1]
    ref, _, _, _ = attend64(q[some], vis[some], codes[:, some] if B > 1 else codes, exps[:, some] if B > 1 else exps,
                            block, d ** -0.5)
    assert abs(drift_of(np64(out[some]), ref)) < 2.0 ** -10, drift_of(np64(out[some]), ref)


RISING = [  # B, Q, n_q, n_kv, d, N, rows: whole items and items that CTAs share
    (1, 592, 64, 4, 64, 131072, 256), (1, 500, 64, 4, 64, 131072, 256), (1, 592, 64, 4, 128, 131072, 256),
    (1, 500, 64, 4, 128, 98304, 256), (1, 296, 64, 4, 256, 131072, 128), (1, 250, 64, 4, 256, 131072, 128),
    (37, 2, 8, 4, 64, 1 << 19, 16)]


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("case", RISING, ids=[f"d{c[4]}-Q{c[1]}-N{c[5]}-rows{c[6]}" for c in RISING])
def test_attend_bf16_parts_under_a_rising_reference(case, weights):
    """Logits that rise with the slot: the sums of earlier parts count, scaled down."""
    B, Q, n_q, n_kv, d, N, rows = case
    block = 64
    g = torch.Generator(device=DEV).manual_seed(10)
    codes = torch.randint(0x30, 0x50, (2, B, n_kv, N, d), generator=g, device=DEV, dtype=torch.uint8)
    codes[0, ..., 0] = torch.linspace(-440.0, 440.0, N, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
    exps = torch.full((2, B, n_kv, N // block), 125, dtype=torch.uint8, device=DEV)
    q = 0.02 * torch.randn(B * Q, n_q, d, generator=g, device=DEV)
    q[..., 0] = 4.0 * d ** 0.5 / 110.0    # logits from -4 to 4
    q = q.to(torch.bfloat16)
    vis = (N - torch.arange(B * Q, device=DEV) % 100).to(torch.int32)
    vis[1], vis[B * Q - 2] = 40000, 0
    acc = torch.zeros(B, n_kv, N // block, device=DEV) if weights else None
    p = bd.kv8_params(n_q, n_kv, d, block, N, "bf16")
    out = torch.full_like(q, float("nan"))
    with rows_of_a_cta(rows):
        bd.csa_kv8_attend(p, q, vis, codes[0], exps[0], codes[1], exps[1], out, acc=acc)
    if B == 1:
        some = torch.tensor([0, 1, 2, Q // 2, Q - 2, Q - 1], device=DEV)
        ref, _, mag, load = attend64(q[some], vis[some], codes, exps, block, d ** -0.5)
    else:
        some = torch.tensor([0, 1, 34, 35, 72, 73], device=DEV)
        b = some[::2] // Q
        ref, _, mag, load = attend64(q[some], vis[some], codes[:, b], exps[:, b], block, d ** -0.5)
    within(np64(out[some]), ref, attend_tol("bf16", d, N, ref, mag, load, load.max()), "out")
    if weights:   # each row's weights add up to 1, summed in fp32 over its slots and the rows
        rows_seen = (vis.view(B, Q) > 0).sum(1).double().cpu().numpy()[:, None] * (n_q // n_kv)
        eps = (2 * d + 24) * U * load.max()
        within(np64(acc).sum(-1), np.broadcast_to(rows_seen, (B, n_kv)),
               (2 * eps + (N / 8 + 2 * block + Q * n_q // n_kv + 24) * U) * rows_seen, "acc")


@pytest.mark.parametrize("case", [c for c in FORMS if c[2] > 3 and c[6] == 160] + [("bf16", 1, 250, 64, 4, 256, 160, 128)],
                         ids=lambda c: f"{c[0]}-d{c[5]}-rows{c[7]}")
def test_attend_weights_that_vanish_are_zero(case):
    """The first block takes everything, by 2^200, and has the largest value
    exponent; slots that weigh nothing, visible or masked, add nothing to acc."""
    act, B, Q, n_q, n_kv, d, N, rows = case
    g = torch.Generator().manual_seed(11)
    block = 16
    codes = ordinary_codes((2, B, n_kv, N, d), g, 1.0)
    codes[0, ..., 0] = 0
    codes[0, :, :, :block, 0] = 0x70          # 128
    exps = torch.full((2, B, n_kv, N // block), 127, dtype=torch.uint8)
    exps[1], exps[1, :, :, 0] = 87, 167
    q = 0.1 * torch.randn(B * Q, n_q, d, generator=g)
    q[..., 0] = 200.0 / 128 * np.log(2.0) * d ** 0.5
    q, codes, exps = q.to(DT[act]).to(DEV), codes.to(DEV), exps.to(DEV)
    vis = (block + 1 + torch.arange(B * Q, device=DEV) % (N - block)).to(torch.int32)
    acc = torch.zeros(B, n_kv, N // block, device=DEV)
    out = run_form(case, codes, exps, q, vis, block, d ** -0.5, acc=acc)
    assert (acc[..., 0] - Q * n_q // n_kv).abs().max() < 1e-3 * Q * n_q // n_kv
    assert acc[..., 1:].max() < 1e-45
    ref, _, mag, load = attend64(q, vis, codes, exps, block, d ** -0.5)
    within(np64(out), ref, attend_tol(act, d, N, ref, mag, load, load.max()) + N * 2.0 ** -32 * 448 * 2.0 ** 40, "out")


# ------------------------------------------------------- long calls side by side --
LONG = [  # act, B, Q, n_q, n_kv, d, block, N: sums in tensor memory, in memory, calls that run as several
    ("f32", 37, 1, 8, 4, 128, 64, 16384), ("bf16", 1, 250, 64, 4, 128, 64, 98304),
    ("bf16", 5, 500, 64, 8, 64, 16, 16384), ("f32", 1, 287, 64, 8, 64, 32, 6144)]


def test_long_calls_captured_and_on_streams_of_their_own():
    """Calls in parts, captured with a workspace each and replayed at the same time,
    give the bits of the same calls alone."""
    runs = []
    for i, (act, B, Q, n_q, n_kv, d, block, N) in enumerate(LONG):
        g = torch.Generator(device=DEV).manual_seed(12 + i)
        p = bd.kv8_params(n_q, n_kv, d, block, N, act)
        codes = torch.randint(0, 0x58, (2, B, n_kv, N, d), generator=g, device=DEV, dtype=torch.uint8)
        exps = torch.full((2, B, n_kv, N // block), 121, dtype=torch.uint8, device=DEV)
        q = (0.3 * torch.randn(B * Q, n_q, d, generator=g, device=DEV)).to(DT[act])
        vis = (N - torch.arange(B * Q, device=DEV) % 300).to(torch.int32)
        acc = torch.zeros(B, n_kv, N // block, device=DEV)
        ws = torch.empty(bd.kv8_attend_workspace_bytes(p, B, Q, True), dtype=torch.uint8, device=DEV)
        out, want, wacc = torch.empty_like(q), torch.empty_like(q), acc.clone()

        def call(o, a, w=None, p=p, q=q, vis=vis, codes=codes, exps=exps):
            bd.csa_kv8_attend(p, q, vis, codes[0], exps[0], codes[1], exps[1], o, acc=a, decay=0.5, workspace=w)
        call(want, wacc)
        s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=s):
            call(out, acc, ws)
        # (the graph reads these tensors at every replay: they have to live as long)
        runs.append((s, graph, out, acc, want, wacc, (q, vis, codes, exps, ws)))
    torch.cuda.synchronize()
    for _ in range(3):
        for s, graph, out, acc, *_ in runs:
            with torch.cuda.stream(s):
                acc.zero_()
                graph.replay()
    torch.cuda.synchronize()
    for _, _, out, acc, want, wacc, _ in runs:
        assert torch.equal(out, want) and torch.equal(acc, wacc)

