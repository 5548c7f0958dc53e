"""What the step's calls refuse is refused alike by both forms of the binding."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import mla_latent_cache_attention_gb300 as mod
    mod.lib()
    return mod


@pytest.mark.parametrize("plain", [True, False])
@pytest.mark.parametrize("width", [0, 1, 63, 514])
def test_rope_of_a_width_that_is_no_rotation(m, monkeypatch, plain, width):
    if not plain:
        monkeypatch.setattr(m, "_step", m._DeclinedStep)
    q = torch.zeros((2, 4, 1024), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="even width from 2 to 512"):
        m.rope(q, torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros((8, width), device="cuda"))
