"""The closed form by which shares of latent attention are found, against sums over row tiles: compiled for the host (no GPU)."""
import subprocess

from paged_kv_cache_279_gb300 import build

PROGRAM = r"""
#include <stdio.h>
#include "latent_tc.cuh"
using namespace pkv::latent;

template <int N, int TOK, bool ONE>
long check(int H, int L, int n, int max_q, bool decode) {
    const int32_t lens[1] = {L}, starts[2] = {0, n};
    Args a{};
    a.lens = lens, a.q_starts = decode ? nullptr : starts;
    a.S = 1, a.T = n, a.H = H, a.B = 16, a.maxb = 1 << 26, a.max_len = 1 << 30, a.max_q = max_q;
    int l = 0;
    while (1 << l < H) ++l;
    a.hshift = 31 + l, a.hmul = (uint32_t)((1ull << a.hshift) / (unsigned)H + 1);
    Walk<N, TOK, ONE> w;
    w.open(a, 0);
    long bad = 0;
    int64_t sum = 0;
    for (int k = w.k0; k < w.R; ++k) {
        // tokens that the last row of row tile k sees, from the definition
        const int nq = n < max_q ? n : max_q, rows = nq * H, last = (k + 1) * N < rows ? (k + 1) * N - 1 : rows - 1;
        int see = decode ? L : L - n + last / H + 1;
        see = see < 0 ? 0 : see > L ? L : see;
        const int tiles = (see + TOK - 1) / TOK;
        bad += tiles != w.tiles(a, k) || tiles < 1;
        if constexpr (!ONE) bad += w.before(a, k) != sum;
        for (int64_t off = sum; off < sum + tiles + kHead; ++off) {
            int64_t at = off;
            w.find(a, at);
            bad += w.k != k || at != off - sum;
        }
        sum += tiles + kHead;
    }
    bad += w.total(a) != sum;
    return bad;
}

template <int N, int TOK, bool ONE>
long all() {
    long bad = 0;
    const int heads[] = {1, 2, 3, 5, 16, 33, 64, 100, 127, 128}, lens[] = {0, 1, 47, 48, 49, 64, 127, 128, 129, 300, 1000, 70000};
    for (int H : heads)
        for (int L : lens) {
            bad += H <= N ? check<N, TOK, ONE>(H, L, 1, 1, true) : 0;
            for (int n : {0, 1, 2, 3, 7, 40, 129, 500})
                for (int more : {0, 1})  // fewer queries attended than there are
                    if (!ONE || (n - more) * H <= N) bad += n - more < 1 ? 0 : check<N, TOK, ONE>(H, L, n, n - more, false);
        }
    return bad;
}

int main() {
#ifdef UNEVEN
    Walk<32, 48, false> w{};
    Args a{};
    return (int)w.before(a, 1);
#else
    const long bad = all<128, 128, false>() + all<16, 48, true>() + all<32, 48, true>() + all<16, 64, true>() + all<32, 64, true>() + all<64, 64, true>() + all<64, 128, false>();
    printf("%ld\n", bad);
    return bad != 0;
#endif
}
"""


def _compile(tmp_path, *flags):
    src, exe = tmp_path / "walk.cu", tmp_path / "walk"
    src.write_text(PROGRAM)
    return exe, subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-I", build.CSRC, "-I", build.INCLUDE, *flags, str(src), "-o", str(exe)],
                               capture_output=True, text=True)


def test_closed_form(tmp_path):
    exe, r = _compile(tmp_path)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def test_row_tiles_that_do_not_divide_a_tile_have_none(tmp_path):
    _, r = _compile(tmp_path, "-DUNEVEN")
    assert r.returncode != 0 and "the closed form" in r.stderr
