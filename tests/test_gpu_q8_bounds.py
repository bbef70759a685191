"""The 8-bit cache and the rotation at the ends of their ranges, on the GPU, against
64-bit references."""
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
