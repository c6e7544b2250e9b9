"""The arithmetic by which mk_attn.cu cuts its work, run on the host from the same header.

The join finds an item's partial results by the workers of its first and last tile, so every
worker in between has to have a tile of it; and the cost of a sequence's blocks is a closed
form that has to agree with the walk over them."""
import os
import subprocess

import persistent_moe_decode_sm_gb300 as mk

HERE = os.path.dirname(os.path.abspath(__file__))


def test_the_cut_owns_every_tile_once_and_without_gaps(tmp_path):
    exe = str(tmp_path / "cut")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I", mk.CSRC,
                           os.path.join(HERE, "attn_cut_check.cpp"), "-o", exe])
    r = subprocess.run([exe], stdout=subprocess.PIPE, timeout=300)
    assert r.returncode == 0, r.stdout.decode()
    assert r.stdout.decode().strip() == "ok"
