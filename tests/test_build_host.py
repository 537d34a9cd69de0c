"""The build and the binding's extension module (no GPU): the C library does
not depend on the module, and no module outlives the headers it was made from."""
import os
import shutil

import pytest

from exact_attention_33_gb300 import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A source tree of one empty unit, built in tmp_path with nvcc; `command`
    stands for the module's compiler."""
    src = tmp_path / "csrc"
    src.mkdir()
    (src / "a.cu").write_text("extern \"C\" int fa_nothing() { return 0; }\n")
    (src / "torch_calls.cpp").write_text("// the module\n")
    for name, value in (("CSRC", src), ("BUILD", tmp_path / "_build"),
                        ("BUILD_CHECKED", tmp_path / "_build_checked"),
                        ("LIB", tmp_path / "libfa.so"), ("LIB_CHECKED", tmp_path / "libfa_checked.so"),
                        ("TORCH_CALLS", tmp_path / "_torch_calls.so")):
        monkeypatch.setattr(b, name, str(value))
    monkeypatch.setattr(b, "SOURCES", ["a.cu"])
    monkeypatch.setattr(b, "torch_calls_command",
                        lambda out: ["cp", str(src / "torch_calls.cpp"), out])
    return tmp_path


def age(path, seconds):
    st = os.stat(path)
    os.utime(path, (st.st_atime, st.st_mtime - seconds))


def test_library_without_the_module(tree, monkeypatch):
    """A module that does not compile leaves the library as the nvcc build made
    it, says so, and leaves no older module behind."""
    (tree / "_torch_calls.so").write_text("older headers")
    age(tree / "_torch_calls.so", 10 ** 9)
    monkeypatch.setattr(b, "torch_calls_command", lambda out: ["false"])
    with pytest.warns(RuntimeWarning):
        assert b.build() == str(tree / "libfa.so")
    assert (tree / "libfa.so").exists() and not (tree / "_torch_calls.so").exists()

    def no_torch(out):
        raise ImportError("torch")
    monkeypatch.setattr(b, "torch_calls_command", no_torch)
    with pytest.warns(RuntimeWarning):
        b.build(force=True)


def test_checked_build_renews_the_module(tree):
    (tree / "csrc" / "torch_calls.cpp").write_text("old")
    b.build(checked=True)
    assert (tree / "_torch_calls.so").read_text() == "old"
    (tree / "csrc" / "torch_calls.cpp").write_text("new")
    for f in ("libfa_checked.so", "_torch_calls.so"):
        age(tree / f, 60)
    b.build(checked=True)
    assert (tree / "_torch_calls.so").read_text() == "new"


def test_a_lost_module_is_made_again(tree):
    b.build()
    os.remove(tree / "_torch_calls.so")
    age(tree / "libfa.so", 0)
    before = os.stat(tree / "libfa.so").st_mtime_ns
    b.build()
    assert (tree / "_torch_calls.so").exists()
    assert os.stat(tree / "libfa.so").st_mtime_ns == before   # not linked again


def test_a_module_that_does_not_load(tmp_path, monkeypatch):
    """The calls are then made from Python."""
    import exact_attention_33_gb300 as fa
    b.build()
    fa.load_library()
    (tmp_path / "_torch_calls.so").write_text("made for another torch")
    monkeypatch.setattr(fa, "_PKG", str(tmp_path))
    monkeypatch.setattr(fa, "_calls", None)
    with pytest.warns(RuntimeWarning):
        assert fa._short() is False
    assert fa._short() is False
    shutil.rmtree(tmp_path)
    torch = pytest.importorskip("torch")
    q = torch.zeros((1, 8, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.fa_fwd_window(q, q, q, 4)
