"""Row arithmetic of the 8-bit cache's append, compiled for the host: the rows that a
span has in each block of the grid, up to the largest cache (no GPU)."""
import subprocess

from gist_token_chunk_b200 import build

MAIN = r"""
#include "%s/ssa_q8_cache.cuh"
#include <cstdio>
int main() {
    long long n, t, r, start, count;
    while (scanf("%%lld %%lld %%lld %%lld %%lld", &n, &t, &r, &start, &count) == 5) {
        // the blocks that the call's grid has for a sequence
        const long long most = (t + r - 2) / r + 1, have = n / r, blocks = most < have ? most : have;
        const ssa_q8::FastDiv by_rows((uint32_t)r);
        long long rows = 0, wild = 0, next = start;
        for (long long i = 0; i < blocks; ++i) {
            int lo = 0, hi = 0;
            const long long blk = (long long)by_rows.div((uint32_t)start) + i;
            if (!ssa_q8::rows_in_block((int)start, (int)count, blk, (int)r, lo, hi)) continue;
            wild += lo != next || hi > start + count || lo / r != blk || (hi - 1) / r != blk;
            next = hi;
            rows += hi - lo;
        }
        printf("%%lld %%lld\n", rows, wild);
    }
}
"""

LARGEST = 2 ** 31 - 1025


def test_rows_of_every_block(tmp_path):
    """Each row of the span in one block and in order, none outside it; padded calls (count
    under T) at the end of the largest caches, where later blocks begin past 2^31."""
    cases = []
    for n, r in ((LARGEST // 64 * 64, 64), (LARGEST // 256 * 256, 256), (LARGEST, 1),
                 (LARGEST // 100 * 100, 100), (2 ** 30, 2 ** 23), (96, 32), (37, 1)):
        for t in (1, 10000, 100000):
            for count in (0, 1, 30, min(t, n)):
                if count <= min(t, n):
                    for start in (0, n // 2 - count // 2, n - count):
                        cases.append((n, t, r, start, count))
    # more blocks in the grid than rows are left, one row a block
    cases.append((LARGEST, 3000000, 1, LARGEST - 5, 5))
    src = tmp_path / "spans.cu"
    src.write_text(MAIN % build.CSRC)
    exe = tmp_path / "spans"
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-o", str(exe), str(src)], check=True)
    text = "\n".join(" ".join(map(str, c)) for c in cases) + "\n"
    out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
    got = [tuple(map(int, line.split())) for line in out.splitlines()]
    assert len(got) == len(cases)
    for c, (rows, wild) in zip(cases, got):
        assert (rows, wild) == (c[4], 0), c
