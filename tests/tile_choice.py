"""The tile sizes that the library's launches choose, asked of its own estimate
(csrc/tile_choice.h) through a small program, tests/c/tile_choice.cpp."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_ffn_moe_amd", "csrc")


class Tiles:
    def __init__(self, folder):
        self.exe = os.path.join(str(folder), "tile_choice")
        cc = subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC,
                             os.path.join(ROOT, "tests", "c", "tile_choice.cpp"), "-o", self.exe], capture_output=True, text=True)
        assert cc.returncode == 0, cc.stderr

    def ask(self, questions):
        run = subprocess.run([self.exe], input="\n".join(questions) + "\n", capture_output=True, text=True, timeout=120)
        assert run.returncode == 0, run.stderr
        return [tuple(int(v) for v in line.split()) for line in run.stdout.splitlines()]

    def sizes(self, dtype):
        v = self.ask([f"sizes {dtype}"])[0]
        return list(zip(v[::2], v[1::2]))


def launches(dtype, T, H, Is):
    """Questions for the tiled products of the shared expert: its two projections (in training and with adapters),
    and the two launches of the backward pass."""
    return dict(w13=f"product {dtype} {T} {2 * Is} {H}", down=f"product {dtype} {T} {H} {Is}",
                d_gu=f"pair {dtype} {T} {Is} {H} {H} {Is} {T}", d_x=f"pair {dtype} {T} {H} {2 * Is} {2 * Is} {H} {T}")
