"""The native binding belongs to the serving calls alone, and to the torch it was built against."""
import os
import shutil

import pytest
import torch

import context_gqa_attention_gb300 as cpa
from context_gqa_attention_gb300 import _build


@pytest.fixture
def fresh(monkeypatch, tmp_path):
    """The package as a new process finds it, its binding's files in a folder of this test's own."""
    _build.build()
    binding, built_for = tmp_path / "cpattn_binding.so", tmp_path / "cpattn_binding.txt"
    shutil.copy(_build.BUILT_FOR, built_for)
    monkeypatch.setattr(_build, "BINDING", str(binding))
    monkeypatch.setattr(_build, "BUILT_FOR", str(built_for))
    monkeypatch.setattr(cpa, "_LIB", None)
    monkeypatch.setattr(cpa, "_BINDING", None)
    return binding, built_for


def _others_work_and_serving_refuses(match):
    assert cpa.cp_decode_plan(2, 2, 1, 8, 16, 100)[0] >= 1      # one of the calls that do without
    x = torch.zeros(2, 2, 64)
    for _ in range(2):
        with pytest.raises(cpa.CPError, match=match):
            cpa.cp_kv_cache_read(x, x, x, x, x, 1, 8)


def test_without_the_binding(fresh):
    _others_work_and_serving_refuses("missing")
    assert not _build.up_to_date()


def test_with_a_file_that_does_not_load(fresh):
    fresh[0].write_bytes(b"not a library")
    _others_work_and_serving_refuses("does not load")


def test_with_the_binding_of_another_torch(fresh):
    fresh[0].write_bytes(b"not looked at")
    fresh[1].write_text(_build.binding_target().replace(torch.__version__, "1.0"))
    _others_work_and_serving_refuses("was built for torch 1.0")
    assert not _build.up_to_date()


def test_as_it_was_built():
    _build.build()
    assert _build.up_to_date() and os.path.exists(_build.BINDING) and _build.binding_built_for() == _build.binding_target()
    assert cpa._binding() is cpa._binding()
