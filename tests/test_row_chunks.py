"""Which 16-byte chunks the norm of unaligned rows moves whole (csrc/row_chunks.h): every chunk that
reaches outside its matrix is left to element accesses, and no other one. Compiled for the host; the
matrices are small enough to go through all of them, rows of fewer than 16 bytes among them."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "expert_routing_grouped_layer_b200", "csrc")
SOURCE = r"""
#include <cstdio>
#include "row_chunks.h"
int main() {
    long chunks = 0, outside = 0;
    for (int es = 2; es <= 4; es += 2)
        for (int base = 0; base < 16; base += es)
            for (int H = 1; H <= 20; ++H)
                for (int ld = H; ld <= H + 9; ++ld)
                    for (int T = 1; T <= 11; ++T) {
                        const long m = 4096 + base, first = m, last = m + ((long)(T - 1) * ld + H) * es;
                        for (int t = 0; t < T; ++t) {
                            const long row = m + (long)t * ld * es;
                            const moe::RowChunks r(row, first, last, H * es);
                            const long from = row - r.off;
                            if (from % 16 || r.off < 0 || r.off > 15 || r.end - r.off != H * es) return 1;
                            for (int c = 0; c < r.end; c += 16) {
                                const bool in = from + c >= first && from + c + 16 <= last;
                                if (in != r.whole(c)) return 2;
                                ++chunks;
                                outside += !in;
                            }
                        }
                    }
    printf("%ld %ld", chunks, outside);
}
"""


def test_chunks_that_move_whole_lie_inside_the_matrix(tmp_path):
    src, exe = tmp_path / "chunks.cpp", tmp_path / "chunks"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0
    chunks, outside = map(int, out.stdout.split())
    assert 0 < outside < chunks
