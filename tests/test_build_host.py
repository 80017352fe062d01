"""What build() makes where torch is missing, changed or not to be compiled against: compilers are stand-ins."""
import os

import pytest
import torch

from context_attention_dits_gb300 import build


@pytest.fixture
def made(tmp_path, monkeypatch):
    """Commands that build() runs, into a folder of its own; made.fails names a source that does not compile."""
    for name, at in (("PKG", "."), ("LIBDIR", "lib"), ("LIB", "lib/libcpattn.so"), ("BIND", "lib/_cpbind.so")):
        monkeypatch.setattr(build, name, str(tmp_path / at), raising=False)

    class Made(list):
        fails = None

        def run(self, cmd):
            self.append(cmd)
            if any(os.path.basename(x) == self.fails for x in cmd):
                return 1, "no such header"
            with open(cmd[cmd.index("-o") + 1], "w"):
                return 0, ""

        def of(self, source):
            return sum(any(os.path.basename(x) == source for x in cmd) for cmd in self)

    made = Made()
    monkeypatch.setattr(build, "_run", made.run)
    return made


def test_library_without_torch(made, monkeypatch):
    import importlib.util
    import sys
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: None)
    monkeypatch.setitem(sys.modules, "torch", None)   # import torch: ImportError
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert made.of("bind.cpp") == 0


def test_library_stays_where_the_marshalling_does_not_compile(made):
    made.fails = "bind.cpp"
    with pytest.raises(RuntimeError, match="no such header"):
        build.build()
    assert os.path.exists(build.LIB)


def test_nothing_is_made_twice(made):
    build.build()
    n = len(made)
    assert made.of("bind.cpp") == 1 and n > len(build.SOURCES)
    build.build()
    assert len(made) == n


def test_marshalling_of_another_torch(made, monkeypatch):
    build.build()
    n = made.of("rope.cu")
    monkeypatch.setattr(torch, "__version__", "9.9.9+cu999")
    build.build()
    assert made.of("bind.cpp") == 2 and made.of("rope.cu") == n   # made for it, and nothing else again
    monkeypatch.undo()


def test_marshalling_by_the_abi_of_torch(made):
    build.build()
    command = next(cmd for cmd in made if any(x.endswith("bind.cpp") for x in cmd))
    assert f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}" in command
