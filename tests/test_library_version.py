"""A library that is older than the binding is told as such, whether its version differs or
it lacks an entry point."""

import types

import pytest

from sparse_moe_transformer_route_b200 import binding as B
from tests.test_abi import built_library  # noqa: F401


def _library(version, lacks=()):
    names = {n: (lambda *a: 0) for n in B.EXPORTS if n not in lacks}
    names["moe_abi_version"] = lambda: version
    return types.SimpleNamespace(**names)


@pytest.mark.parametrize("version,lacks,told", [
    (B.ABI_VERSION - 1, ("moe_grouped_gemm", "moe_grouped_gemm_wgrad"), f"ABI {B.ABI_VERSION - 1}, this binding ABI"),
    (B.ABI_VERSION + 1, (), f"ABI {B.ABI_VERSION + 1}, this binding ABI"),
    (B.ABI_VERSION, ("moe_grouped_gemm", "moe_quantize_microscaled"), "lacks moe_grouped_gemm, moe_quantize_microscaled"),
])
def test_an_older_library_says_to_rebuild(monkeypatch, version, lacks, told):
    monkeypatch.setattr(B, "_lib", None)
    monkeypatch.setattr(B.ctypes, "CDLL", lambda path: _library(version, lacks))
    with pytest.raises(RuntimeError, match=told) as err:
        B.lib()
    assert "rebuild with" in str(err.value)
    assert B._lib is None


def test_the_built_library_loads(monkeypatch):
    monkeypatch.setattr(B, "_lib", None)
    assert B.lib().moe_abi_version() == B.ABI_VERSION
