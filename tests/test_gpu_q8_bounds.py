"""The 8-bit cache and the rotation at the ends of their ranges, on the GPU, against
64-bit references."""
import functools
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import q8_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gist_token_chunk_b200 import ssa as mod

    return mod


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append ---

def test_append_at_the_end_of_the_largest_cache(ssa):
    """A padded call (T far over count) whose later blocks begin past 2^31: the span is
    written, its neighbours and every other row that is looked at stay."""
    R, d, T, n = 64, 64, 10000, 100
    N = (2 ** 31 - 1025) // R * R
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < N * d + (4 << 30):
        pytest.skip("needs 142 GB of device memory")
    code = torch.empty(1, 1, N, d, dtype=torch.uint8, device="cuda")
    scale = torch.full((1, 1, N // R), 2.0, device="cuda")
    code[:, :, -4096:] = 9
    code[:, :, :20000] = 9
    x = torch.randn(1, 1, T, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    start = N - n
    ssa.ssa_cache_append_q8(x.cuda(), None, i32([start]), code, None, scale, None, count=i32([n]))
    assert ssa.ssa_cache_get_status() == 0
    want, ws = np.full((1, 1, 128, d), 9, np.uint8), np.full((1, 1, 2), 2.0, np.float32)
    q8_ref.append(x.double().numpy(), want, ws, R, [128 - n], [n])
    assert np.array_equal(q8_ref.TABLE[code[:, :, -128:].cpu().numpy()], q8_ref.TABLE[want])
    assert np.array_equal(scale[:, :, -2:].cpu().numpy(), ws)
    assert bool((code[:, :, -4096:-128] == 9).all()) and bool((code[:, :, :20000] == 9).all())
    assert bool((scale[:, :, :-2] == 2.0).all())
    k, _ = ssa.ssa_cache_read_q8(code, None, scale, None, i32([start]), T, count=i32([n]),
                                 dtype=torch.float32)
    assert np.array_equal(k[:, :, :n].cpu().double().numpy(), q8_ref.values(want, ws, R)[:, :, -n:])
    assert not bool(k[:, :, n:].any())
    del code, scale
    torch.cuda.empty_cache()


# ------------------------------------------------------------- status word ---

def test_two_readers_of_the_status_word(ssa):
    """Two threads read on streams of their own: an error reaches exactly one of them."""
    import threading

    x = torch.ones(1, 1, 1, 64, device="cuda", dtype=torch.bfloat16)
    c = torch.zeros(1, 1, 8, 64, dtype=torch.uint8, device="cuda")
    s = torch.ones(1, 1, 1, device="cuda")
    bad, rounds = i32([9]), 400
    got = [[], []]
    gate = threading.Barrier(2)

    def read(i):
        stream = torch.cuda.Stream()
        for _ in range(rounds):
            if i == 0:
                ssa.ssa_cache_append_q8(x, None, bad, c, None, s, None)
                torch.cuda.synchronize()
            gate.wait(60)
            got[i].append(ssa.ssa_cache_get_status(stream))
            gate.wait(60)

    threads = [threading.Thread(target=read, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got[0]) == len(got[1]) == rounds
    err = ssa.SSA_ERR_DEVICE_STATUS
    assert all(sorted(p) == [0, err] for p in zip(*got))


# ------------------------------------------------------------------ decode ---
#
# What the decode may be off by, for each output on its own (u = 2^-24): a logit is off by
# e = (d/8 + 8) u A, A = max over rows of sum |q_i k_i| / sqrt(d). The same weights are summed
# and averaged, so that moves an output by e sum w |v - out|; the exponential and the weights'
# 22 bits, the additions (rows / 64 + 8 of 2 u) add a share of sum w |v|. A weight times its
# value scale is held to 2^-32 of the largest such product, and a weight under 2^-126 of the
# largest may be taken as zero.

def spread_reference(x, case, b, j, sel):
    """Outputs of one (sequence, KV head) for a selection, and the bound of each."""
    B, Hq, Hkv, d, n_max, C, g, topk, lens, dtype = case
    G, n = Hq // Hkv, lens[b]
    M = n // C
    q = x["q"][b, j * G:(j + 1) * G].double().numpy()
    mine = np.asarray([m for m in sel if m >= 0], np.int64)
    keep = np.ones(M, bool)
    keep[mine] = False
    raw = np.concatenate([np.arange(m * C, m * C + C) for m in mine] + [np.arange(M * C, n)]).astype(np.int64)
    gist = np.repeat(keep, g).nonzero()[0]

    def rows(name):
        code = np.concatenate([q8_ref.TABLE[x[f"{name}_gist"][b, j][gist]], q8_ref.TABLE[x[f"{name}_raw"][b, j][raw]]])
        s = np.concatenate([x[f"{name}_gist_scale"][b, j][gist // g], x[f"{name}_raw_scale"][b, j][raw // C]])
        return code, s.astype(np.float64)[:, None]

    (kc, ks), (vc, vs) = rows("k"), rows("v")
    lx = q @ (kc * ks).T / np.sqrt(d)
    w = np.exp(lx - lx.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    v = vc * vs
    out = w @ v
    e = (d / 8 + 8) * U * (np.abs(q) @ np.abs(kc * ks).T).max(1, keepdims=True) / np.sqrt(d)
    off = np.stack([(w[h][:, None] * np.abs(v - out[h])).sum(0) for h in range(G)])
    tol = e * off * 1.01 + (w @ np.abs(v)) * (2.0 ** -20 + (len(v) / 64 + 8) * 2 * U)
    floor = 2.0 ** -32 * (w * vs.T).max(1, keepdims=True) + 2.0 ** -125 * vs.T
    return out, tol + floor @ np.abs(vc)


U = 2.0 ** -24


def check_spread(ssa, x, case):
    from test_gpu_q8 import gpu_args

    B, Hq, Hkv, d, n_max, C, g, topk, lens, dtype = case
    G = Hq // Hkv
    out, sel = ssa.ssa_decode_q8(*gpu_args(x, case))
    assert ssa.ssa_cache_get_status() == 0
    out, sel = out.cpu().double().numpy(), sel.cpu().numpy()
    for b in range(B):
        for j in range(Hkv):
            ref, tol = spread_reference(x, case, b, j, sel[b, j])
            err = np.abs(out[b, j * G:(j + 1) * G] - ref)
            assert (err <= tol).all(), (b, j, (err / np.maximum(tol, 1e-300)).max(), err.max())


SPREAD = [
    (1, 4, 1, 64, 1024, 64, 8, 4, (1000,), "bf16"),
    (1, 8, 1, 128, 1024, 64, 8, 4, (1000,), "fp32"),
    (2, 4, 2, 64, 16384, 64, 8, 16, (16300, 5000), "bf16"),   # many splits
    (1, 12, 1, 128, 8192, 128, 8, 8, (8100,), "bf16"),        # two head groups
]


@functools.lru_cache(maxsize=None)
def made_once(case):
    from test_gpu_q8 import decode_inputs

    return decode_inputs(case, seed=30)


def inputs(case):
    return {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in made_once(case).items()}


def sharp_inputs(case, logit, place):
    """Queries along one dim each, and for each head one row, at `place`, with that logit; all
    others 0. Values at random."""
    B, Hq, Hkv, d, n_max, C, g, topk, lens, dtype = case
    G = Hq // Hkv
    x = inputs(case)
    x["q"] = torch.zeros(B, Hq, d)
    for h in range(Hq):
        x["q"][:, h, h % G] = logit * d ** 0.5 / 256
    x["q"] = x["q"].to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    for n in ("k_raw", "k_gist"):
        x[n][:] = 0
        x[n + "_scale"][:] = 1.0
    for b in range(B):
        M = lens[b] // C
        for h in range(G):
            # the ties of the scores select the first chunks: chunk 1 is selected, M - 2 is not
            if place == "raw":
                x["k_raw"][b, :, C + 3 * h + 1, h] = 0x78  # 256
            elif place == "gist":
                x["k_gist"][b, :, (M - 2) * g + h % g, h] = 0x68  # 64: under the first chunks'
                x["k_gist"][b, :, :topk * g, h] = 0x68
            else:
                x["k_raw"][b, :, lens[b] - 1 - h, h] = 0x78
    return x


@pytest.mark.parametrize("place", ["raw", "gist", "tail"])
@pytest.mark.parametrize("case", SPREAD)
def test_decode_weight_on_a_block_of_small_values(ssa, case, place):
    """A head whose weight lies on one row of a block whose value scale is far under another
    visible block's: the row's value to its own precision."""
    B, Hq, Hkv, d, n_max, C, g, topk, lens, dtype = case
    for logit, up in ((40, 12), (40, 20), (40, 30), (40, 40), (40, 60), (100, 100)):
        x = sharp_inputs(case, logit * (4 if place == "gist" else 1), place)
        for b in range(B):
            M = lens[b] // C
            for n in ("v_raw", "v_gist"):
                x[n + "_scale"][b, :, :M + (n == "v_raw")] = 2.0 ** -20
                x[n + "_scale"][b, :, M // 2] = 2.0 ** (up - 20)
            x["v_raw_scale"][b, :, 2] = 2.0 ** (up - 20)
        check_spread(ssa, x, case)


@pytest.mark.parametrize("loud", [0.1, 1.0, 8.0])
@pytest.mark.parametrize("case", SPREAD)
def test_decode_value_scales_at_random(ssa, case, loud):
    """Value scales over 80 powers of two, also of blocks beside each other."""
    x = inputs(case)
    x["q"] = x["q"] * loud
    rnd = np.random.RandomState(int(loud * 10))
    for n in ("v_raw_scale", "v_gist_scale"):
        x[n] = np.where(np.isnan(x[n]), x[n], np.ldexp(1.0, rnd.randint(-40, 41, x[n].shape))).astype(np.float32)
    check_spread(ssa, x, case)


@pytest.mark.parametrize("step", [3.0, 30.0, -3.0])
@pytest.mark.parametrize("case", SPREAD)
def test_decode_logits_climb_while_values_shrink(ssa, case, step):
    """Each chunk's logits `step` above the last one's and its values as much smaller, so that
    all chunks count in the sums of the outputs and only the last in the softmax's."""
    B, Hq, Hkv, d, n_max, C, g, topk, lens, dtype = case
    x = inputs(case)
    x["q"] = x["q"].clone()
    M = n_max // C
    x["q"][:] = 0
    x["q"][:, :, 0] = d ** 0.5
    for n in ("k_raw", "k_gist"):
        x[n][:, :, :, 0] = 0x38  # 1
        x[n][:, :, :, 1:] = 0
        x[n + "_scale"][:] = (abs(step) * (np.arange(M) + 1 if step > 0 else M - np.arange(M))).astype(np.float32)
    for n in ("v_raw_scale", "v_gist_scale"):
        at = np.arange(M) if step > 0 else np.arange(M)[::-1]
        x[n][:] = np.ldexp(1.0, np.clip(60 - np.round(abs(step) * at * 1.4427), -100, 60).astype(int)).astype(np.float32)
    check_spread(ssa, x, case)


@pytest.mark.parametrize("size", [1e6, 1e9, 1e12])
@pytest.mark.parametrize("case", SPREAD)
def test_decode_logits_past_24_bits(ssa, case, size):
    """A logit so large that fp32 does not hold its sum with a scale's exponent: the output is the
    row's value, whatever its scale."""
    for place in ("raw", "tail"):
        x = sharp_inputs(case, 256.0, place)
        for n in ("k_raw_scale", "k_gist_scale"):
            x[n][:] = np.float32(size / 256.0)
        for n in ("v_raw_scale", "v_gist_scale"):
            x[n][:] = 2.0 ** -9
        check_spread(ssa, x, case)


@pytest.mark.parametrize("case", SPREAD)
def test_decode_values_at_the_ends_of_fp32(ssa, case):
    """Value scales of 2^-100, 2^100 and none that is a power of two, each alone and side by side."""
    for scales in ((2.0 ** -100,), (2.0 ** 100,), (2.0 ** -100, 2.0 ** 100), (1.37e-12, 2.9e5, 0.71)):
        x = inputs(case)
        for n in ("v_raw_scale", "v_gist_scale"):
            at = np.arange(x[n].shape[2])
            x[n][:] = np.asarray(scales, np.float32)[at % len(scales)]
        check_spread(ssa, x, case)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_decode_an_infinite_query_selects_by_its_sign(ssa, dtype, sign):
    """One head's query has an infinite element: chunks with a gist key of its sign there score
    +inf, the first of them are selected, and the other heads' outputs are as defined."""
    from test_gpu_q8 import gpu_args

    case = (1, 3, 1, 64, 2048, 32, 4, 6, (2000,), dtype)
    x = inputs(case)
    x["q"] = x["q"].clone()
    x["q"][0, 1, 5] = sign * float("inf")
    M, g = 2000 // 32, 4
    rnd = np.random.RandomState(3)
    code = np.where(rnd.rand(M, g) < 0.06, 0x30, 0xb0)  # 0.5, -0.5
    code[7] = 0xb0
    code[7, 2] = 0  # the product is NaN, which no maximum takes
    x["k_gist"][0, 0, :M * g, 5] = code.ravel()
    score = np.where(code == 0, -np.inf, sign * np.where(code == 0x30, np.inf, -np.inf)).max(1)
    other = [x["q"][0, h].double().numpy() for h in (0, 2)]
    keys = q8_ref.values(x["k_gist"][0, 0][None, None, :M * g], x["k_gist_scale"][0, 0][None, None, :M], g)[0, 0]
    score = np.maximum(score, np.stack([keys @ q for q in other]).max(0).reshape(M, g).max(1))
    want = np.sort(np.lexsort((np.arange(M), -score))[:6])
    out, sel = ssa.ssa_decode_q8(*gpu_args(x, case))
    assert np.array_equal(sel[0, 0].cpu().numpy(), want)
    x["q"][0, 1] = 0.0
    ref, tol = spread_reference(x, case, 0, 0, sel[0, 0].cpu().numpy())
    out = out[0].cpu().double().numpy()
    assert np.isnan(out[1]).all() and (np.abs(out - ref) <= tol)[[0, 2]].all()


# ---------------------------------------------------------------- rotation ---

def exact_turn(pos, freqs):
    """Cosines and sines of pos * f, the product and its reduction exact, [rows, pairs]."""
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    c, s = np.empty((len(pos), len(freqs))), np.empty((len(pos), len(freqs)))
    for i, p in enumerate(pos):
        for j, f in enumerate(freqs):
            w = Fraction(int(p)) * Fraction(float(f))
            w = float(w - round(w / two_pi) * two_pi)
            c[i, j], s[i, j] = math.cos(w), math.sin(w)
    return c, s


@pytest.mark.parametrize("half", [True, False])
def test_rope_angles_at_every_position(ssa, half):
    """The rotation of unit pairs is the cosine and sine themselves, at near, far and the
    farthest positions: the fraction in half turns is rounded to fp32 (2^-25, so pi / 2 u of
    angle), sincospi is off by a step (u), the products are exact."""
    rnd = np.random.RandomState(2)
    pos = np.concatenate([np.arange(-3, 40), rnd.randint(0, 1 << 20, 60), rnd.randint(1 << 29, 2 ** 31 - 1, 60),
                          2 ** 31 - 1 - np.arange(60), -2 ** 31 + np.arange(10)])
    freqs, _ = ssa.ssa_rope_freqs(64, 10000.0)
    c, s = exact_turn(pos, freqs.tolist())
    i = np.arange(32)
    a, b = (i, i + 32) if half else (2 * i, 2 * i + 1)
    q = torch.zeros(1, 2, len(pos), 64)
    q[:, 0, :, a] = 1.0
    q[:, 1, :, b] = 1.0
    layout = ssa.SSA_ROPE_HALF if half else ssa.SSA_ROPE_INTERLEAVED
    for inverse in (False, True):
        y, _ = ssa.ssa_rope(q.cuda(), None, i32(pos[None].tolist()), freqs.cuda(), layout, inverse=inverse)
        y = y[0].cpu().double().numpy()
        t = -s if inverse else s
        for got, want in ((y[0][:, a], c), (y[0][:, b], t), (y[1][:, a], -t), (y[1][:, b], c)):
            assert np.abs(got - want).max() <= 2.6 * U, np.abs(got - want).max() / U


# ------------------------------------------------------------ host threads ---

def test_other_threads_run_while_a_launch_waits(ssa):
    """Calls into a stream whose queue is full wait for room; the process's other threads do not."""
    import threading
    import time

    x = torch.zeros(1, 1, 1, 64, device="cuda", dtype=torch.bfloat16)
    c = torch.zeros(1, 1, 8, 64, dtype=torch.uint8, device="cuda")
    s = torch.ones(1, 1, 1, device="cuda")
    zero, stream = i32([0]), torch.cuda.Stream()
    ssa.ssa_cache_append_q8(x, None, zero, c, None, s, None)
    torch.cuda.synchronize()
    gaps, stop = [], threading.Event()

    def tick():
        last = time.monotonic()
        while not stop.is_set():
            time.sleep(0.005)
            now = time.monotonic()
            gaps.append(now - last)
            last = now

    ticker = threading.Thread(target=tick)
    ticker.start()
    try:
        with torch.cuda.stream(stream):
            torch.cuda._sleep(3_000_000_000)  # about 1.5 s
        t0 = time.monotonic()
        for _ in range(3000):
            ssa.ssa_cache_append_q8(x, None, zero, c, None, s, None, stream=stream)
        waited = time.monotonic() - t0
        torch.cuda.synchronize()
    finally:
        stop.set()
        ticker.join()
    assert waited > 0.8, "the queue was never full"
    assert max(gaps) < 0.4, max(gaps)
