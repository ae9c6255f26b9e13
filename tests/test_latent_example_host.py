"""The latent attention layer of examples/ on the CPU, with its operators stubbed: whose workspace a
step of it uses."""
import importlib.util
import os

import torch


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "latent_layer.py")
    spec = importlib.util.spec_from_file_location("latent_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_steps_share_no_workspace_of_the_layers(monkeypatch):
    """Steps of one layer may run at the same time, on two streams or in two graphs: they share partial
    sums only where their caller passes both the same workspace."""
    example = load()
    given = []

    class Stub:
        @staticmethod
        def latent_append(*x, **k):
            pass

        @staticmethod
        def latent_decode_workspace(*x, **k):
            return torch.empty(64, dtype=torch.uint8)

        @staticmethod
        def latent_decode(q, *x, workspace=None, **k):
            given.append(workspace)
            return torch.zeros(*q.shape[:2], example.LATENT, dtype=q.dtype), None

    monkeypatch.setattr(example, "sk", Stub)
    layer = example.LatentLayer(64, 2, device="cpu")
    cache = example.PagedCache(3, 40, page=16, device="cpu")
    x, lens = torch.zeros(3, 64, dtype=torch.bfloat16), torch.tensor([5, 1, 40], dtype=torch.int32)
    for _ in range(2):
        assert layer.attend_step(x, cache, lens).shape == (3, 2, example.HEAD)
    assert given[0] is None or given[0] is not given[1]
    kept = torch.empty(64, dtype=torch.uint8)
    layer.attend_step(x, cache, lens, workspace=kept)
    assert given[2] is kept
    assert not any(isinstance(v, dict) and v for v in vars(layer).values())
