"""build() from several callers at once: one compiles, the others wait for its library."""
import concurrent.futures
import os
import time

from lora_moe_gb300 import build


def test_one_caller_builds(tmp_path, monkeypatch):
    monkeypatch.setattr(build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    running, seen = [0], []

    def fake(verbose, ptxas_info):
        running[0] += 1
        seen.append(running[0])
        time.sleep(0.2)
        with open(build.LIB, "w"):
            pass
        running[0] -= 1

    monkeypatch.setattr(build, "_build", fake)
    with concurrent.futures.ThreadPoolExecutor(4) as ex:
        paths = list(ex.map(lambda _: build.build(), range(4)))
    assert seen == [1] and set(paths) == {build.LIB} and os.path.exists(build.LIB)
    with concurrent.futures.ThreadPoolExecutor(3) as ex:   # asked for outright: each, in turn
        list(ex.map(lambda _: build.build(force=True), range(3)))
    assert seen == [1, 1, 1, 1]
