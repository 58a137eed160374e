"""What the build makes, in which order, and when again. CPU only; no compiler runs."""

import os

import pytest

from jagged_pointwise_attention_b200 import _native, build as b


def test_the_built_binding_carries_its_tag():
    b.build()
    assert not b.binding_needs_build()
    assert _native.serving().__doc__ == b.binding_tag()


def test_the_binding_is_rebuilt_for_another_torch(tmp_path, monkeypatch):
    out = tmp_path / "_serving.so"
    assert b.binding_needs_build(str(out))
    out.write_bytes(b"\x7fELF" + b.binding_tag().encode() + b"\0rest")
    assert not b.binding_needs_build(str(out))
    monkeypatch.setattr("torch.__version__", "2.99.0+cu999")
    assert b.binding_needs_build(str(out))
    out.write_bytes(b"\x7fELF" + b.binding_tag().encode() + b"\0rest")
    assert not b.binding_needs_build(str(out))
    os.utime(out, (1, 1))                       # older than its source
    assert b.binding_needs_build(str(out))


def test_the_library_is_built_where_the_binding_cannot_be(monkeypatch, tmp_path):
    made = []
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libhstu.so"))
    monkeypatch.setattr(b, "build_library", lambda force, verbose, out, extra: made.append(out) or out)

    def no_headers(force=False):
        raise OSError("no torch headers")
    monkeypatch.setattr(b, "build_binding", no_headers)
    with pytest.raises(OSError):
        b.build(out=b.LIB)
    assert made == [b.LIB]
    assert b.build(out=str(tmp_path / "other.so")) == str(tmp_path / "other.so")
