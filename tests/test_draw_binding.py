"""What the binding of the draws refuses before a call (no GPU needed: tensors are stood in for)."""
import pytest

torch = pytest.importorskip("torch")

import diffusion_drafter_draft_gb300 as dd  # noqa: E402


@pytest.mark.parametrize("key", ["accepted_len", "path", "bonus"])
def test_outputs_on_another_device(monkeypatch, key):
    monkeypatch.setattr(dd, "_need", lambda *a: 0)             # (it wants CUDA tensors)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    tree = dict(tok=i(2, 5), par=i(2, 5), depth=i(2, 5), n_nodes=i(2))
    out = dict(accepted_len=i(2), path=i(2, 3), bonus=i(2))
    out[key] = out[key].to("meta")
    with pytest.raises(ValueError, match=f"{key} must be on cpu"):
        dd.verify_filtered(tree, torch.zeros(2, 5, 8), dd.ROWS_PER_NODE, 3, torch.zeros(2, 5), out=out)
