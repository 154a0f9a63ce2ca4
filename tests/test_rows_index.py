"""The row kernels' index arithmetic (csrc/rows_index.h), enumerated on the host."""
import subprocess

from combine_persistent_warp_gb300 import build

PRELUDE = '#include <cstdio>\n#include <initializer_list>\n#include "rows_index.h"\nusing namespace cpw;\n'


def _run(tmp_path, body):
    src, exe = tmp_path / "check.cpp", tmp_path / "check"
    src.write_text(PRELUDE + "int main() {\n" + body + "\nreturn 0; }\n")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I" + build.CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_rows_that_are_zeroed_stay_inside_whatever_the_offsets_hold(tmp_path):
    """Block b of `blocks` walks the rows rest_begin() + b, + blocks, ... below M."""
    _run(tmp_path, """
    const int ends[] = {-2147483647 - 1, -7, 0, 1, 29, 30, 31, 1 << 30, 2147483400, 2147483647};
    const int sizes[] = {0, 1, 30, 1 << 30};
    for (int M : sizes)
        for (int total : ends) {
            const int first = rest_begin(total, M);
            if (first < 0 || first > M) { printf("M %d, offsets[E] %d: from row %d on\\n", M, total, first); return 1; }
            for (int blocks : {1, 152, 2048})
                for (int b = 0; b < blocks; ++b)
                    if (static_cast<long long>(first) + b > 2147483647LL) { printf("M %d, offsets[E] %d, block %d: past 31 bits\\n", M, total, b); return 1; }
            if (total >= 0 && total <= M && first != total) return 1;
        }
    """)


def test_shifted_vectors_are_read_from_inside_the_matrix(tmp_path):
    """Whatever the leads of the written and of the read rows, the two aligned vectors that hold elements
    e .. e + V - 1 lie inside the matrix wherever the kernels load them: where `inside` holds for the
    vector, or the row is `amid` the matrix."""
    _run(tmp_path, """
    for (int V : {4, 8})
        for (int H = 1; H <= 70; ++H) {
            const int rim = rim_of(H, V), vectors = vectors_of(H, V);
            for (int lead = 0; lead < V; ++lead)                      // of the written row
                if (vectors * V - lead < H) { printf("H %d V %d: elements left over\\n", H, V); return 1; }
            for (int rows : {1, 2, 2 * rim, 2 * rim + 1, 2 * rim + 3})
                for (int r = 0; r < rows; ++r)
                    for (int g = 0; g < vectors; ++g) {
                        if (!inside(g, H, V) && !amid(r, rows, rim))
                            continue;
                        for (int lead = 0; lead < V; ++lead)
                            for (int past = 0; past < V; ++past) {    // the read row's elements past a boundary
                                const int e = g * V - lead, at = past + e, start = (at + 64 * V) / V * V - 64 * V;
                                const long long lo = static_cast<long long>(r) * H + start - past, hi = lo + 2 * V;
                                if (lo < 0 || hi > static_cast<long long>(rows) * H) {
                                    printf("V %d H %d, row %d of %d, vector %d, leads %d and %d: elements %lld .. %lld of %lld\\n", V, H, r, rows, g,
                                           lead, past, lo, hi, static_cast<long long>(rows) * H);
                                    return 1;
                                }
                            }
                    }
        }
    """)
