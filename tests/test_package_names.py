"""Names of the package that are looked up when they are used (no GPU)."""

import int8_quantized_matmul_absmax_amd as i8


def test_an_op_that_is_replaced_is_found(monkeypatch):
    """A program that wraps an op of `ops` wraps it for the package, too, whether it has
    been used before or not."""
    for name in ("beam_select", "kv_pages_step", "workspace_bytes", "MAX_BEAM_COUNT"):
        assert getattr(i8, name) is getattr(i8.ops, name)
        other = object()
        with monkeypatch.context() as m:
            m.setattr(i8.ops, name, other)
            assert getattr(i8, name) is other
        assert getattr(i8, name) is getattr(i8.ops, name)
