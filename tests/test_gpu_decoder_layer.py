"""The example decoder layer: append, attention and the routed-expert FFN as a
serving step runs them, prompts and captured decode steps."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_layer_attends_over_what_it_appended(lib, example):
    from tests.test_gpu_kv import plain_attention, table_of_codes
    prompts, steps = [70, 1, 33], 3
    layer, outputs = example.run(prompts, steps)
    assert lib.moe_read_device_status(layer.err) == (lib.MOE_OK, 0)
    assert layer.kv_len.tolist() == [p + steps for p in prompts]
    assert all(torch.isfinite(y).all() for y in outputs)

    class Cache:                      # what the plain attention wants to know of the last step
        heads, total, new = layer.kv_heads, layer.kv_len.tolist(), [1] * len(prompts)
        cu = torch.arange(len(prompts) + 1)

        def values(self, b, which, upto):
            codes, scale = (layer.k, layer.ks) if which == "k" else (layer.v, layer.vs)
            ids = layer.table[b, : -(-upto // codes.shape[2])].long()
            x = table_of_codes()[codes[ids].long()] * scale[ids].double()[:, :, None, None]
            return x.transpose(0, 1).reshape(self.heads, -1, layer.dim)[:, :upto]

    q, got = layer.last
    ref, mag, _ = plain_attention(Cache(), q, layer.dim ** -0.5, 0, 0.0, False)
    # the bound of tests/test_gpu_kv.py
    assert ((got.double() - ref).abs() <= (2.0 ** -11 + 2.0 ** -14) * (mag + ref.abs()) + 2.0 ** -8 * ref.abs() + 1e-7).all()


def test_layer_repeats_bit_for_bit(example):
    first, second = example.run([64, 30], 2), example.run([64, 30], 2)
    assert len(first[1]) == 3
    for x, y in zip(first[1], second[1]):
        assert torch.equal(x, y)
