"""Row counts near 2^31 (csrc/rows.h), on the CPU: the header is compiled for the host with
overflow of signed numbers trapped, and walked at the ends of the range against 64 bits."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_qmv_quantize_gb300", "csrc")

PROGRAM = r"""
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include "rows.h"

int main()
{
    const int most = 0x7fffffff;
    int wrong = 0;
    const int counts[] = {1, 2, 15, 16, 17, 31, 32, 1215, 1216, 1217, 7300, most - 2433, most - 1216, most - 17, most - 1, most};
    for (int M : counts) {
        for (int n : {1, 2, 16}) wrong += qmv::groups_of(M, n) != (static_cast<int64_t>(M) + n - 1) / n;
        for (int m = M > 70 ? M - 70 : 0; m < M; ++m)
            for (int ahead = 0; ahead < 40; ++ahead) wrong += qmv::row_ahead(m, ahead, M) != (static_cast<int64_t>(m) + ahead < M);
        for (int step : {1, 3, 173, 608, 1216}) {
            if (step > M) continue;
            for (int first = 0; first < step; first += step > 200 ? 101 : 1) {
                // the last rows of the walk that begins with `first`, as a CTA's
                int64_t want = first + (static_cast<int64_t>(M - first - 1) / step > 5 ? static_cast<int64_t>(M - first - 1) / step - 5 : 0) * step;
                qmv::RowsInTurn at{static_cast<unsigned>(want), step, M - static_cast<int>(want)};
                for (; at.ahead(0); at.next(), want += step) {
                    for (int n = 0; n <= 2; ++n) {
                        wrong += at.ahead(n) != (want + static_cast<int64_t>(n) * step < M);
                        if (at.ahead(n)) wrong += at.row(n) != want + static_cast<int64_t>(n) * step;
                    }
                }
                wrong += want < M;
            }
        }
    }
    std::printf("%d\n", wrong);
    return wrong != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_rows_up_to_the_largest_count(tmp_path):
    source, program = tmp_path / "rows.cpp", tmp_path / "rows"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-Wall", "-Werror", f"-I{CSRC}", str(source), "-o", str(program)], check=True)
    r = subprocess.run([str(program)], capture_output=True, text=True)
    assert (r.returncode, r.stdout.strip()) == (0, "0")


def test_the_appends_compare_rows_by_what_is_left():
    """No sum of a row and an offset is compared with the number of rows: it passes 2^31 for the largest."""
    text = open(os.path.join(CSRC, "norm_rope.cu")).read()
    assert "< g.M" not in text and "(g.M +" not in text
