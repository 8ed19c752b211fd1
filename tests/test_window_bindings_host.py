"""The Python side of the rotary append's and the windowed attention's bindings, without a GPU."""
import os
import sys

import pytest


@pytest.fixture(scope="module")
def native():
    from paged_kv_cache_207_gb300 import build, _native
    build.build()
    return _native


def test_bounds_past_int32_stay_on_their_side(native):
    for x, want in ((-2**32 + 5, -2**31), (-2**63, -2**31), (-2**31, -2**31), (-7, -7), (0, 0), (2**31 - 1, 2**31 - 1),
                    (2**31, 2**31 - 1), (2**32 + 5, 2**31 - 1), (2**100, 2**31 - 1)):
        assert native._bound(x) == want, x


@pytest.fixture()
def small_build(monkeypatch, tmp_path):
    """A build of one source into a folder of its own."""
    from paged_kv_cache_207_gb300 import build
    monkeypatch.setattr(build, "SOURCES", ["pa_block_manager.cpp"])
    for name, file in (("LIB", "lib.so"), ("QUICK", "_quick.so"), ("BUILD", "objects")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    if not build._has_headers():
        pytest.skip("no headers of Python or torch: the binding is not compiled")
    return build


def test_build_takes_a_compiler_with_arguments(small_build, monkeypatch, tmp_path):
    fake = tmp_path / "compiler.py"
    fake.write_text("import sys\nopen(sys.argv[sys.argv.index('-o') + 1], 'w').write(' '.join(sys.argv[1:]))\n")
    monkeypatch.setenv("CXX", f"{sys.executable} {fake} --first")
    assert small_build.build() == small_build.LIB and os.path.exists(small_build.LIB)
    assert open(small_build.QUICK).read().startswith("--first ")
    assert not small_build._stale(small_build.LIB) and not small_build._stale(small_build.QUICK)


@pytest.mark.parametrize("compiler", ["false", "/no/such/compiler"])
def test_build_does_without_the_compiled_binding(small_build, monkeypatch, tmp_path, compiler, capfd):
    monkeypatch.setenv("CXX", compiler)
    (tmp_path / "_quick.so").write_text("of other sources")
    assert small_build.build(force=True) == small_build.LIB and os.path.exists(small_build.LIB)
    assert not os.path.exists(small_build.QUICK) and "pa_binding.cpp" in capfd.readouterr().err
    # the library is not built again for the binding's sake
    at = os.stat(small_build.LIB).st_mtime_ns
    small_build.build()
    assert os.stat(small_build.LIB).st_mtime_ns == at
