"""Sizes beyond 31 bits are refused, not taken by their low 32 bits."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_sizes_beyond_31_bits():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import diffusion_drafter_draft_gb300 as dd
    dd.lib()
    V = 2 ** 32 + 64                                           # (8.6 GB of bf16, of which only the head is written)
    x = torch.empty(V, dtype=torch.bfloat16, device="cuda")
    x[:64] = 0.0
    u = torch.zeros(1, device="cuda")
    with pytest.raises(dd.DartreeError) as e:
        dd.sample(x.view(1, V), u)
    assert e.value.code == dd.EUNSUPPORTED
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    tree = dict(tok=i(1, 2), par=i(1, 2), depth=i(1, 2), n_nodes=i(1))
    with pytest.raises(dd.DartreeError) as e:
        dd.verify_filtered(tree, x.view(1, 1, V), dd.ROWS_PER_POSITION, 1, u.view(1, 1))
    assert e.value.code == dd.EUNSUPPORTED
    del x
    torch.cuda.empty_cache()
