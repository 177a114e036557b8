"""The serving example end to end: a packed prefill and a draft-tree step through the package's calls.
A drafted token's attention equals that of the same tokens run as a prompt: both paths round
weights and output to bf16 (2^-8 each, of values that are averages of N(0, 1) rows: below 2 in
magnitude), so they differ by less than 4 * 2^-8 * 2."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_serve_layer_example():
    spec = importlib.util.spec_from_file_location("serve_layer", os.path.join(ROOT, "examples", "serve_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    r = mod.run()
    assert r["prefill"].shape == (377, 1024) and torch.isfinite(r["prefill"].float()).all()
    assert 0 < r["n_sel"] < 377
    assert torch.isfinite(r["decode"].float()).all() and all(0 < n < r["d_ff"] for n in r["n_active"])
    got, ref = r["decode_attention"][[1, 2, 3]].float(), r["as_prompts"].float()
    assert ref.abs().max() < 2.0
    assert (got - ref).abs().max() <= 4 * 2.0 ** -8 * 2.0
