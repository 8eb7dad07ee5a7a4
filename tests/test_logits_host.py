"""Host-side helpers of the logits calls, without a GPU: compiled with g++ and
compared with the plain definition; and the refusals that rest on them."""
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def compiled(tmp_path, text):
    src, exe = tmp_path / "probe.cpp", tmp_path / "probe"
    src.write_text('#include "ws_host.h"\n#include <cstdio>\n' + text)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "post_processing_gb300", "csrc"),
                    str(src), "-o", str(exe)], check=True)
    return str(exe)


@pytest.fixture(scope="module")
def B():
    import __graft_entry__
    __graft_entry__.build()
    from post_processing_gb300 import binding
    return binding


def share(d, sa, sb, rows, cols):
    a = {r * sa + j for r in range(rows) for j in range(cols)}
    return any(d + s * sb + j in a for s in range(rows) for j in range(cols))


def test_rows_overlap(tmp_path):
    exe = compiled(tmp_path, r'''
int main() {
    long long d, sa, sb, rows, cols, size;
    while (scanf("%lld %lld %lld %lld %lld %lld", &d, &sa, &sb, &rows, &cols, &size) == 6)
        printf("%d\n", (int)ws::rows_overlap((void*)0x100000000ull, sa, (void*)(0x100000000ull + d * size), sb, rows, cols, (size_t)size));
}''')
    g = random.Random(3)
    cases = []
    for _ in range(6000):
        rows, cols = g.randint(1, 5), g.randint(1, 6)
        sa = cols + g.randint(0, 8)
        sb = sa if g.random() < 0.5 else cols + g.randint(0, 8)
        cases.append((g.randint(-5 * sb - 8, 5 * sa + 8), sa, sb, rows, cols, g.choice([2, 4])))
    # the halves of one buffer, rows of a wide one, offsets past 32 bits
    cases += [(100, 200, 200, 8, 100, 4), (-100, 200, 200, 8, 100, 2), (99, 200, 200, 8, 100, 4), (1, 200, 200, 1, 100, 2),
              (100, 200, 400, 3, 100, 4)]
    text = "\n".join(" ".join(map(str, c)) for c in cases)
    got = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.split()
    want = [share(d, sa, sb, rows, cols) for d, sa, sb, rows, cols, _ in cases]
    assert [x == "1" for x in got] == want
    assert 0.2 < sum(want) / len(want) < 0.8
    far = [(3 << 33, 1 << 34, 1 << 34, 6, 1 << 30, 2), ((3 << 33) + (1 << 33), 1 << 34, 1 << 34, 6, 1 << 30, 2)]
    got = subprocess.run([exe], input="\n".join(" ".join(map(str, c)) for c in far), capture_output=True, text=True, check=True).stdout.split()
    assert got == ["0", "1"]


def test_gradients_that_overlap_the_logits_are_refused(B):
    """Before anything is enqueued (the addresses are nobody's)."""
    x = 1 << 20
    for dtype, size in ((B.WS_DTYPE_F32, 4), (B.WS_DTYPE_BF16, 2)):
        # (elements from the logits on, gradient's stride) for 4 rows of 100, 120 apart
        for d, stride in ((1, 120), (-1, 120), (99, 120), (21, 120), (120, 120), (-360, 120), (459, 120), (0, 121), (119, 119),
                          (-300, 101)):
            desc = B.ws_logprobs_desc(4, 100, 120, dtype, B.WS_INDEX_I64, 0, 1.0)
            assert B.ws_logprobs_backward(desc, x, 64, 64, 64, 64, 64, x + d * size, stride, 0) == B.WS_ERR_INVALID_ARGUMENT
            assert "grad_logits" in B.ws_last_error()
            desc = B.ws_distill_desc(4, 100, 120, stride, dtype, B.WS_INDEX_I32, 5, B.WS_DISTILL_TAIL, 1.0)
            assert B.ws_distill(desc, x, 64, 64, 64, 64, x + d * size, 0) == B.WS_ERR_INVALID_ARGUMENT
            assert "grad_logits" in B.ws_last_error()
        # one row: strides do not matter
        desc = B.ws_distill_desc(1, 100, 1000, 700, dtype, B.WS_INDEX_I32, 5, B.WS_DISTILL_TAIL, 1.0)
        assert B.ws_distill(desc, x, 64, 64, 64, 64, x + 7 * size, 0) == B.WS_ERR_INVALID_ARGUMENT


def test_each_query_counts_for_itself(tmp_path):
    """A query that fails leaves the others' answers; answers are kept once the queries could be prepared, and not before."""
    exe = compiled(tmp_path, r'''
int main() {
    ws::AskedOnce<3, 5> t;
    int prepared = 0, queries = 0;
    auto show = [&] {
        for (auto& row : t.of) for (int n : row) printf("%d ", n);
        printf("%d %d %d\n", (int)t.asked, prepared, queries);
    };
    auto query = [&](int a, int b, int* n) {
        ++queries;
        *n = 77;                          // what a failed query leaves there does not count
        if (b == 4 || (a == 0 && b == 1)) return false;
        *n = 10 * a + b + 1;
        return true;
    };
    t.ask([&] { ++prepared; return false; }, query);
    show();
    t.ask([&] { ++prepared; return true; }, query);
    show();
    t.ask([&] { ++prepared; return true; }, query);
    show();
}''')
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split("\n")
    kept = "1 0 3 4 0 11 12 13 14 0 21 22 23 24 0"
    assert out[0].strip() == "0 " * 15 + "0 1 0"
    assert out[1].strip() == kept + " 1 2 15"
    assert out[2].strip() == kept + " 1 2 15"
