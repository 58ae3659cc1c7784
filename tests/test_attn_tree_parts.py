"""How fp4_attn_tree shares keys and workgroups, on the host: the parts of trees' keys against the launch and the scratch
that are planned for them, and launches of every size within the device's limits."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def test_parts_and_launches(tmp_path):
    exe = str(tmp_path / "tree_parts_check")
    subprocess.run(["g++", "-O2", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-std=c++17", "-o", exe,
                    os.path.join(HERE, "pins", "tree_parts_check.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr
    assert int(r.stdout.split()[1]) > 1000                 # calls whose keys are cut
