"""The prompt kernel's search for its tile, run on the CPU: the source's own functions, compiled for
the host, with a warp's 32 lanes taken in turn.  Every unit (a tile's tokens) of every sequence
is found by one index and by no other, the indexes behind the last find none, and there are never more units
than the grid has room for, whatever the starts hold."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "bit_plane_select_gb300", "csrc", "trit_attn_prompt.cu")

# A collective is met by every lane: each leaves its value, the lanes are taken in turn until all have, and each
# then reads.  Two sets of values, so that a lane may go on to the next one before the others have read.
HOST = r"""
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <ucontext.h>
#include "trit.h"
#define __device__
#define __forceinline__ inline
using std::max;
using std::min;
constexpr int kBlockKeys = 128;
static ucontext_t lanes[32], home;
static char stacks[32][65536];
static int now, turn[32];
static int64_t values[2][32];
static const int64_t *meet(int64_t v) {
    int64_t *all = values[turn[now]++ & 1];
    all[now] = v;
    swapcontext(&lanes[now], &home);
    return all;
}
static int __shfl_up_sync(unsigned, int v, int o) { const int64_t *a = meet(v); return int(a[now >= o ? now - o : now]); }
static int __shfl_sync(unsigned, int v, int who) { const int64_t *a = meet(v); return int(a[who & 31]); }
static unsigned __ballot_sync(unsigned, bool v) {
    const int64_t *a = meet(v);
    unsigned r = 0;
    for (int i = 0; i < 32; ++i) r |= a[i] ? 1u << i : 0u;
    return r;
}
static bool __any_sync(unsigned, bool v) { return __ballot_sync(~0u, v) != 0; }
static unsigned __reduce_add_sync(unsigned, unsigned v) {
    const int64_t *a = meet(v);
    unsigned r = 0;
    for (int i = 0; i < 32; ++i) r += unsigned(a[i]);
    return r;
}
static unsigned __reduce_max_sync(unsigned, unsigned v) {
    const int64_t *a = meet(v);
    unsigned r = 0;
    for (int i = 0; i < 32; ++i) r = max(r, unsigned(a[i]));
    return r;
}
static int __ffs(int v) { return __builtin_ffs(v); }
static void raise_flag(uint32_t *err, uint32_t bit) { *err |= bit; }
%s
static PromptArgs A;
static int k, found[32];
static bool sorted, report;
static Span spans[32];
static void lane_main() {
    spans[now] = Span{0, 0, 0, 0};
    const int me = now;
    const int unit = sorted ? find_by_length(A, k, me, report, spans[me]) : find_in_order(A, k, me, report, spans[me]);
    found[me] = unit;
    turn[me] = -1;
    for (;;) swapcontext(&lanes[me], &home);
}
int main() {
    static int32_t q[4097], keys[4097];
    static uint32_t err;
    int B, G, by_length, given, last;
    long long q_rows, k_rows;
    while (scanf("%%d %%d %%d %%d %%lld %%lld %%d", &B, &G, &by_length, &given, &q_rows, &k_rows, &last) == 7) {
        for (int i = 0; i <= B; ++i) if (scanf("%%d", q + i) != 1) return 1;
        for (int i = 0; given && i <= B; ++i) if (scanf("%%d", keys + i) != 1) return 1;
        A = PromptArgs();
        A.J.q_starts = q;
        A.J.k_starts = given ? keys : nullptr;
        A.J.q_rows = q_rows;
        A.J.k_rows = k_rows;
        A.J.B = B;
        A.unit = 128 / G;
        A.err = &err;
        err = 0;
        sorted = by_length;
        printf("%%lld", (long long)(q_rows / A.unit + B));
        for (k = 0; k < last; ++k) {
            report = k == 0;
            for (int i = 0; i < 32; ++i) {
                getcontext(&lanes[i]);
                lanes[i].uc_stack.ss_sp = stacks[i];
                lanes[i].uc_stack.ss_size = sizeof stacks[i];
                lanes[i].uc_link = nullptr;
                makecontext(&lanes[i], lane_main, 0);
                turn[i] = 0;
            }
            for (bool left = true; left;) {
                left = false;
                for (now = 0; now < 32; ++now)
                    if (turn[now] >= 0) {
                        swapcontext(&home, &lanes[now]);
                        left = left || turn[now] >= 0;
                    }
            }
            for (int i = 1; i < 32; ++i)
                if (found[i] != found[0] || (found[0] >= 0 && memcmp(&spans[i], &spans[0], sizeof(Span)))) return 2;
            printf(" %%d:%%d:%%d:%%d:%%d", found[0], spans[0].q0, spans[0].nq, spans[0].k0, spans[0].nk);
        }
        printf(" %%u\n", err);
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def search(tmp_path_factory):
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no C++ compiler")
    with open(SRC) as f:
        text = f.read()
    body = re.search(r"(struct PromptArgs \{.*?)\n__device__ __forceinline__ void tma_rows", text, re.S).group(1)
    assert "find_in_order" in body and "find_by_length" in body
    where = tmp_path_factory.mktemp("search")
    src, exe = where / "search.cpp", where / "search"
    src.write_text(HOST % body)
    subprocess.run([cc, "-std=c++17", "-O1", "-w", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)

    def run(q, k, G, by_length, q_rows, k_rows, last):
        """Units that the grid has room for, [(unit, q0, nq, k0, nk)] by index, the flag."""
        B = len(q) - 1
        said = [B, G, int(by_length), int(k is not None), q_rows, k_rows, last, *q, *(k or [])]
        got = subprocess.run([str(exe)], input=" ".join(map(str, said)), check=True, capture_output=True, text=True).stdout.split()
        return int(got[0]), [tuple(map(int, x.split(":"))) for x in got[1:-1]], int(got[-1])
    return run


def starts(n, first=0):
    out = [first]
    for x in n:
        out.append(out[-1] + x)
    return out


def units_of(q, k, G, good):
    unit = 128 // G
    return sorted((u, q[b], q[b + 1] - q[b], k[b], k[b + 1] - k[b]) for b in good for u in range(-(-(q[b + 1] - q[b]) // unit)))


CASES = [
    # queries, keys, query heads to a key head
    ([300, 40], [300, 40], 4),
    ([300, 40], [10, 40], 4),            # more queries than keys, by more than 127 and a unit
    ([5, 400], [5, 100], 4),
    ([700, 5], [0, 5], 4),
    ([159, 3], [1, 3], 4), ([160, 3], [0, 3], 4), ([161, 3], [1, 3], 4), ([192, 3], [0, 3], 4),      # about that border
    ([255, 3], [0, 3], 1), ([256, 3], [0, 3], 1), ([257, 3], [0, 3], 1), ([400, 290], [17, 1], 1),
    ([1, 5, 0, 300], [1000, 5, 40, 777], 4),
    ([90, 41, 0, 0, 500], [0, 0, 0, 7, 200], 7),
    ([12, 3], [0, 200], 128),
    ([(i * 53) % 260 for i in range(32)], [(i * 97) % 330 for i in range(32)], 3),
    ([0, 0, 0], [5, 0, 9], 4),
]


@pytest.mark.parametrize("nq,nk,G", CASES)
@pytest.mark.parametrize("by_length", [False, True])
def test_every_unit_is_found_once(search, nq, nk, G, by_length):
    q, k = starts(nq, 2), starts(nk, 3)
    want = units_of(q, k, G, range(len(nq)))
    room, got, err = search(q, k, G, by_length, q[-1] + 2, k[-1] + 1, len(want) + 3)
    assert len(want) <= room and err == 0
    assert sorted(x for x in got if x[0] >= 0) == want
    assert all(x[0] < 0 for x in got[len(want):])
    if by_length:                        # those with the most blocks first
        unit = 128 // G
        blocks = [max(0, -(-(min((u + 1) * unit, n) + m - n) // 128)) for u, _, n, _, m in got[:len(want)]]
        assert blocks == sorted(blocks, reverse=True)


def test_many_sequences_in_their_order(search):
    nq, nk = [(i * 37) % 90 for i in range(150)], [(i * 11) % 200 for i in range(150)]
    q, k = starts(nq), starts(nk)
    want = units_of(q, k, 4, range(150))
    room, got, err = search(q, k, 4, False, q[-1], k[-1], len(want) + 2)
    assert len(want) <= room and err == 0 and sorted(x for x in got if x[0] >= 0) == want


def apart(q, k, q_rows, k_rows):
    """The sequences that are computed: starts in order and in range, and, once some are not, no rows of one
    before."""
    good, taken, fell = [], 0, False
    for b in range(len(q) - 1):
        ok = 0 <= q[b] <= q[b + 1] <= q_rows and 0 <= k[b] <= k[b + 1] <= k_rows
        fell = fell or not ok
        if ok and q[b + 1] > q[b]:
            assert fell or q[b] >= taken
            if q[b] >= taken:
                good.append(b)
                taken = q[b + 1]
    return good, fell


@pytest.mark.parametrize("by_length", [False, True])
def test_starts_that_fall_leave_the_others_their_tiles(search, by_length):
    """A sequence before the fall keeps its tiles however many the sequences behind it would have."""
    q, k = [0, 20, 500, 100, 480], [0, 20, 500, 100, 480]
    room, got, err = search(q, k, 4, by_length, 500, 500, 40)
    assert [x for x in got if x[0] >= 0 and x[1:] == (0, 20, 0, 20)] == [(0, 0, 20, 0, 20)]
    assert sorted(x for x in got if x[0] >= 0) == units_of(q, k, 4, [0, 1]) and err != 0
    assert all(x[0] < 0 for x in got[room:])


@pytest.mark.parametrize("seed", range(12))
def test_any_starts(search, seed):
    """Starts out of order and out of range: computed sequences are found once, and fit the grid."""
    import random
    rng = random.Random(seed)
    B, G = rng.choice([1, 5, 20, 32, 33, 90]), rng.choice([1, 3, 4, 128])
    q, k = (starts([rng.randrange(300 // G + 2) for _ in range(B)]) for _ in range(2))
    q_rows, k_rows = q[-1] + 1, k[-1] + 1
    for _ in range(seed % 4):
        x = rng.choice([q, q, k])
        x[rng.randrange(B + 1)] = rng.choice([-1, 0, 3, q_rows // 2, q_rows - 1, 2 ** 31 - 1, -2 ** 31])
    good, fell = apart(q, k, q_rows, k_rows)
    want = units_of(q, k, G, good)
    for by_length in (False, True) if B <= 32 else (False,):
        room, got, err = search(q, k, G, by_length, q_rows, k_rows, len(want) + 4)
        assert len(want) <= room and bool(err) == fell
        assert sorted(x for x in got if x[0] >= 0) == want
