"""The build of the Python entry of the serving-step calls: which object it links, and when."""
from __future__ import annotations

import os

from bit_weight_only_pn_gb300 import build


def test_entry_is_linked_for_the_pytorch_in_use(tmp_path, monkeypatch):
    """Built for one PyTorch, for another, and for the first again: the entry is always the present one's."""
    version = ["1"]
    linked = []

    def run(cmd, what):
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write(version[0] if "-c" in cmd else open(next(a for a in cmd if a.endswith(".o"))).read())
        if "-shared" in cmd:
            linked.append(version[0])

    for name, value in (("BUILD", str(tmp_path)), ("BINDING", str(tmp_path / "_step.so")), ("LIBRARY", str(tmp_path / "lib.so")),
                        ("_run", run), ("_torch", lambda: ([], "lib", version[0], 1)), ("nvcc", lambda: "/x/bin/nvcc")):
        monkeypatch.setattr(build, name, value)
    (tmp_path / "lib.so").write_text("")
    os.utime(tmp_path / "lib.so", (0, 0))

    def entry(v):
        version[0] = v
        build._link_binding(build._compile_binding())
        return (tmp_path / "_step.so").read_text()

    assert [entry(v) for v in ("1", "2", "1", "1", "2")] == ["1", "2", "1", "1", "2"]
    assert linked == ["1", "2", "1", "2"]                             # and not again where nothing changed

    # a link that fails leaves no record of an entry that is not there
    def broken(cmd, what):
        raise RuntimeError(what)

    version[0] = "1"
    monkeypatch.setattr(build, "_run", broken)
    try:
        build._link_binding(build._compile_binding())
    except RuntimeError:
        pass
    monkeypatch.setattr(build, "_run", run)
    assert entry("2") == "2" and linked[-1] == "2"


def test_objects_differ_by_python_and_abi(tmp_path, monkeypatch):
    names = set()
    for abi in (0, 1):
        for suffix in ("cpython-312-x86_64-linux-gnu", "cpython-311-x86_64-linux-gnu"):
            monkeypatch.setattr(build, "_torch", lambda: ([], "lib", "1", abi))
            monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: suffix)
            names.add(build._binding_key())
    assert len(names) == 4
