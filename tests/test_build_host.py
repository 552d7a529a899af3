"""The build of the library with a stand-in compiler (no GPU): one source that
does not compile ends the build, and the compilers of the others with it."""

import os
import time

import pytest

from moe_layer_router_amd import build as B

SCRIPT = """#!/bin/sh
for a in "$@"; do
  case "$a" in
    *bad.hip) sleep 0.5; echo "broken" >&2; exit 1;;
    *slow.hip) sleep 60 & echo $! > "{d}/pid"; wait;;
  esac
done
"""


def test_a_failed_source_ends_the_other_compilers(tmp_path, monkeypatch):
    cc = tmp_path / "cc"
    cc.write_text(SCRIPT.format(d=tmp_path))
    cc.chmod(0o755)
    lib = tmp_path / "lib.so"
    monkeypatch.setattr(B, "HIPCC", str(cc))
    monkeypatch.setattr(B, "LIB", str(lib))
    monkeypatch.setattr(B, "SOURCES", [str(tmp_path / "bad.hip"), str(tmp_path / "slow.hip")])
    t0 = time.time()
    with pytest.raises(RuntimeError, match="broken"):
        B.build()
    assert time.time() - t0 < 20 and not lib.exists()
    pid = int((tmp_path / "pid").read_text())
    for _ in range(50):                     # (reparented: gone, or a zombie until it is reaped)
        try:
            state = open(f"/proc/{pid}/stat").read().rsplit(")", 1)[1].split()[0]
        except FileNotFoundError:
            return
        if state == "Z":
            return
        time.sleep(0.1)
    os.kill(pid, 9)
    raise AssertionError("a compiler outlived the build")
