"""Which numbers of a counter are a tile of the recurrence: the check that both of its
kernels make, built for the host."""
import subprocess
from pathlib import Path

CSRC = Path(__file__).resolve().parents[1] / "chunked_gated_delta_kda_amd" / "csrc"


def test_a_counter_that_holds_anything_is_no_tile(tmp_path):
    src, exe = tmp_path / "tiles.cpp", tmp_path / "tiles"
    src.write_text('#include <cstdio>\n#include <cstdlib>\n#include "block_launch.h"\n'
                   "int main(int, char** v) {\n"
                   "    std::printf(\"%d\", (int)kda::is_tile((uint32_t)std::strtoul(v[1], 0, 0), std::atoi(v[2])));\n}\n")
    subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{CSRC}", str(src), "-o",
                    str(exe)], check=True)
    for tiles in (1, 2, 1000, (1 << 25) - 1):
        for number in (0, 1, tiles - 1, tiles, tiles + 1, (1 << 31) - 1, 1 << 31, (1 << 31) + 1, (1 << 32) - tiles,
                       (1 << 32) - 1):
            got = subprocess.run([str(exe), str(number), str(tiles)], capture_output=True, text=True, check=True).stdout
            assert got == str(int(number < tiles)), (number, tiles)


def test_both_kernels_ask_before_they_use_it():
    text = (CSRC / "gated_scan.hip").read_text()
    assert text.count("if (!is_tile(place.order, tiles)) return;") == 2
    for body in text.split("const Place place(a, tiles")[1:]:
        assert body.index("is_tile(place.order, tiles)") < body.index("= place.order")
