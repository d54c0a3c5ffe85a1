"""In which order a piece of an item takes its tiles (csrc/chunk_plan.cuh), on the CPU: each of a
long item's whole tiles once, and no division where no sequence has rows and a share has no units."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_verification_65_gb300", "csrc")

PROGRAM = """
#define __host__
#define __device__
#include "chunk_plan.cuh"
#include <stdio.h>

using spec_attn::piece_turn;

int main()
{
    if (piece_turn(0, 0, 0, 0) != 0 || piece_turn(0, 0, 5, 0) != 0)
        return printf("no units\\n"), 1;
    for (long long per = 1; per < 20; ++per)
        for (int tiles = 0; tiles < 60; ++tiles)
            for (int tile = 0; tile <= tiles; ++tile)
                for (int taken = 0; taken < per; ++taken) {
                    const int turn = piece_turn(taken, tile, tiles, per);
                    const long long back = taken - tile - turn;
                    if (tiles < per ? turn != 0 : turn < 0 || turn >= per || back % per != 0)
                        return printf("%d of %d tiles, %d of %lld taken: %d\\n", tile, tiles, taken,
                                      per, turn), 1;
                }
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_turns(tmp_path):
    source, program = tmp_path / "turns.cpp", tmp_path / "turns"
    source.write_text(PROGRAM)
    # (a division by zero ends the program, on machines too whose instruction for it does not)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=integer-divide-by-zero",
                    "-fsanitize-undefined-trap-on-error", "-I", CSRC, "-o", str(program), str(source)],
                   check=True)
    ran = subprocess.run([str(program)], capture_output=True, text=True)
    assert ran.returncode == 0, (ran.returncode, ran.stdout)
