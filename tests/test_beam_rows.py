"""How the beam selection cuts a row of logits into vectors (csrc/row_cut.h), on the CPU: every
column of rows of any length and place is met once, and no vector reaches outside its row."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_verification_65_gb300", "csrc")

PROGRAM = """
#define __host__
#define __device__
#include "row_cut.h"
#include <stdio.h>
#include <vector>

template <int VEC> int look(int V, int row)
{
    const size_t first = (size_t)row * V;
    const RowCut r = cut_row<VEC>(first, V);
    std::vector<int> met(V, 0);
    const long start = (long)(first / VEC) * VEC;  // the array's element that vector 0 begins with
    for (int v = r.f0; v < r.f1; ++v)
        for (int j = 0; j < VEC; ++j) {
            const long col = start + (long)v * VEC + j - (long)first;
            if (col < 0 || col >= V || col != v * VEC + j - r.mis)
                return printf("V %d row %d: vector %d outside\\n", V, row, v);
            ++met[col];
        }
    const int edges = r.head + V - r.tail;
    if (edges < 0 || edges >= 2 * VEC || r.head < 0 || r.tail < r.head || r.tail > V)
        return printf("V %d row %d: head %d tail %d\\n", V, row, r.head, r.tail);
    for (int i = 0; i < edges; ++i)
        ++met[i < r.head ? i : r.tail + i - r.head];
    for (int c = 0; c < V; ++c)
        if (met[c] != 1)
            return printf("V %d row %d: column %d met %d times\\n", V, row, c, met[c]);
    return 0;
}

int main()
{
    for (int V = 1; V <= 70; ++V)
        for (int row = 0; row < 33; ++row)
            if (look<4>(V, row) || look<8>(V, row))
                return 1;
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_every_column_once(tmp_path):
    source, program = tmp_path / "rows.cpp", tmp_path / "rows"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, "-o", str(program), str(source)],
                   check=True)
    ran = subprocess.run([str(program)], capture_output=True, text=True)
    assert ran.returncode == 0, ran.stdout
