"""How attention cuts the keys of many rows, on the host: the parts of every tile
of rows hold every key that a row sees."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def test_parts_hold_every_key(tmp_path):
    exe = str(tmp_path / "kv_split_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-o", exe, os.path.join(HERE, "pins", "kv_split_check.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr
    assert int(r.stdout.split()[1]) > 100000               # the sweep reaches windows whose keys are cut
