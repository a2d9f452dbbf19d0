"""RouteConfig as the plain value it is (nothing here needs a GPU)."""
import copy
import ctypes
import dataclasses
import io
import pickle

import pytest
import torch

import routing_grouped_expert_gb300 as moe

CONFIGS = [moe.RouteConfig(), moe.RouteConfig("sigmoid", 8, 4, 2, False, 2.5)]


def struct_of(config):
    """What the library is given."""
    c = ctypes.cast(config._ptr, ctypes.POINTER(type(config._c))).contents
    return tuple(getattr(c, name) for name, _ in c._fields_)


@pytest.mark.parametrize("config", CONFIGS, ids=str)
def test_copies_and_pickles(config):
    saved = io.BytesIO()
    torch.save({"config": config}, saved)
    saved.seek(0)
    made = [copy.copy(config), copy.deepcopy(config), copy.deepcopy([config])[0],
            torch.load(saved, weights_only=False)["config"], dataclasses.replace(config)]
    made += [pickle.loads(pickle.dumps(config, p)) for p in range(pickle.HIGHEST_PROTOCOL + 1)]
    for other in made:
        assert other == config and hash(other) == hash(config)
        assert struct_of(other) == struct_of(config)
    assert other._ptr.value != config._ptr.value   # a struct of its own
