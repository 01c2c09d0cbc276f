"""A library built from older sources is refused by its ABI number, before a symbol that it lacks
is looked for (no GPU needed)."""
import os
import re
import shutil
import subprocess

import pytest

from additive_codebook_matmul_amd import _lib, mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# entry points that number 5 had
OLD = _lib.EXPORTED_SYMBOLS


def _older(tmp_path, symbols, version):
    """A library of stubs that reports `version`."""
    source, lib = tmp_path / "older.c", tmp_path / "older.so"
    source.write_text("".join(f"int {name}(void) {{ return {version}; }}\n" for name in symbols))
    subprocess.run([shutil.which("gcc") or "cc", "-shared", "-fPIC", "-o", str(lib), str(source)], check=True)
    return str(lib)


@pytest.mark.parametrize("symbols", [OLD, ("aqlm_abi_version",)], ids=["whole", "few"])
def test_an_older_build_is_refused(monkeypatch, tmp_path, symbols):
    monkeypatch.setattr(_lib, "LIB_PATH", _older(tmp_path, symbols, 5))
    monkeypatch.setattr(_lib, "_lib", None)
    monkeypatch.setattr(mx, "_ready", None)
    with pytest.raises(RuntimeError, match="rebuild"):
        mx._lib()
    assert _lib._lib is None                       # nothing half loaded stays
    with pytest.raises(RuntimeError, match="rebuild"):
        _lib.load_library()


def test_the_number_is_the_header_s():
    text = open(os.path.join(ROOT, "include", "aqlm.h")).read()
    assert int(re.search(r"#define AQLM_ABI_VERSION (\d+)", text).group(1)) == _lib.ABI_VERSION
