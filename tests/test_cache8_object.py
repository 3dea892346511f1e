"""The 8-bit cache's Python object (CPU)."""
import pytest

torch = pytest.importorskip("torch")


def make():
    from head_latent_attention_qkv_gb300 import api
    return api.Cache8(torch.zeros(2, 16, 512, dtype=torch.uint8).view(torch.float8_e4m3fn),
                      torch.zeros(2, 16, 64, dtype=torch.bfloat16), torch.ones(2, 16))


def test_its_tensors_cannot_be_replaced():
    # (its calls use the tensors' addresses, taken once)
    c = make()
    other = make()
    for name in ("latent", "rope", "scale", "num_pages", "page_size", "device_index"):
        was = getattr(c, name)
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(other, name))
        with pytest.raises(AttributeError):
            delattr(c, name)
        assert getattr(c, name) is was or getattr(c, name) == was
    with pytest.raises(AttributeError):
        c.elsewhere = 1
    assert [x.data_ptr() for x in c] == [c.latent.data_ptr(), c.rope.data_ptr(), c.scale.data_ptr()]


def test_its_tensors_must_fit():
    from head_latent_attention_qkv_gb300 import api
    c = make()
    for bad in ((c.latent[:1], c.rope, c.scale), (c.latent, c.rope[:, :8], c.scale), (c.latent, c.rope, c.scale[0]),
                (c.latent, c.rope.half(), c.scale), (c.latent, c.rope, c.scale.double()),
                (c.latent.view(torch.uint8), c.rope, c.scale)):
        with pytest.raises(ValueError):
            api.Cache8(*bad)
