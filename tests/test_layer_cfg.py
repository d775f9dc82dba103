"""LayerCfg stays a plain frozen value whatever calls it went through."""
import copy
import ctypes
import dataclasses
import pickle

import pytest

from bit_expert_ffn_router_b200 import moe as M


def used():
    cfg = M.LayerCfg(d=512, f=256, E=32, k=4, renorm=0)
    assert M.workspace_bytes(cfg, 4) > 0  # as any call does, builds the C structure
    return cfg


def test_a_structure_that_the_caller_changes_changes_no_later_call():
    cfg = used()
    want = M.workspace_bytes(cfg, 4)
    c = cfg.c()
    c.k, c.E = 999, 7
    assert M.workspace_bytes(cfg, 4) == want
    assert (cfg.c().k, cfg.c().E) == (4, 32)


def test_fields_alone_are_held():
    cfg = used()
    assert M.LayerCfg(**vars(cfg)) == cfg
    assert dataclasses.asdict(cfg) == vars(cfg)


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c)), lambda c: c.replace()])
def test_copies(how):
    cfg = used()
    other = how(cfg)
    assert other == cfg and hash(other) == hash(cfg) and other is not cfg
    assert bytes(other.c()) == bytes(cfg.c()) and M.workspace_bytes(other, 4) == M.workspace_bytes(cfg, 4)
    with pytest.raises(dataclasses.FrozenInstanceError):
        other.k = 5


def test_a_changed_copy_has_a_structure_of_its_own():
    cfg = used()
    a, b = M.LayerCfg.ref(cfg)._obj, cfg.replace(k=7).ref()._obj
    assert (a.k, b.k) == (4, 7) and ctypes.sizeof(a) == ctypes.sizeof(b)
