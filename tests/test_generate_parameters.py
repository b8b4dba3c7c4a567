"""The forms in which generate takes its sampling parameters, on the CPU with
stand-ins for the model and the samplers: numbers, tensors and arrays of one
value, and one value per prompt."""
import math

import numpy as np
import pytest
import torch

import test_generate_rows as T
from test_generate_rows import G, R

PROMPTS = [[1, 2, 3], [4, 5]]


def _scalar(logits, temperature, top_p, uniforms, out, stream=None):
    """llama_sample: one temperature and top-p for all rows."""
    for b in range(logits.shape[0]):
        out[b] = R.sample(logits[b], float(torch.tensor(float(temperature))), 0, float(torch.tensor(float(top_p))), 0.0,
                          0.0 if uniforms is None else float(uniforms[b]))
    return out


@pytest.fixture
def run(monkeypatch):
    calls = []
    monkeypatch.setattr(G, "sample", lambda *a, **k: (calls.append("scalar"), _scalar(*a, **k))[1])
    monkeypatch.setattr(G, "sample_rows", lambda *a, **k: (calls.append("rows"), T._rows(*a, **k))[1])
    u = torch.rand(24, 2, generator=torch.Generator().manual_seed(3))

    def go(prompts=PROMPTS, uniforms=u, **kw):
        calls.clear()
        out, _ = G.generate(T._Model(), prompts, max_gen_len=5, uniforms=uniforms, **kw)
        return out, set(calls)
    return go


@pytest.mark.parametrize("wrap", [torch.tensor, np.array, np.float64, lambda x: torch.tensor([x]), lambda x: np.array([x]),
                                  lambda x: torch.tensor([[x]])])
def test_one_value_in_a_tensor_or_array(run, wrap):
    """The scalar sampler's path, as with a number."""
    want, kinds = run(temperature=0.75, top_p=0.875)
    assert kinds == {"scalar"}
    assert run(temperature=wrap(0.75), top_p=wrap(0.875)) == (want, {"scalar"})
    assert run(temperature=wrap(0.75), top_p=0.875) == (want, {"scalar"})
    greedy, _ = run(temperature=0.0)
    assert run(temperature=wrap(0.0)) == (greedy, {"scalar"})


def test_one_value_beside_a_list(run):
    want, kinds = run(temperature=[0.75, 0.75], top_p=[0.875, 0.875], top_k=[7, 7])
    assert kinds == {"rows"}
    assert run(temperature=torch.tensor(0.75), top_p=np.array(0.875), top_k=torch.tensor(7))[0] == want
    assert run(temperature=torch.tensor([0.75, 0.75]), top_p=np.array([0.875, 0.875]), top_k=np.array([7, 7]))[0] == want


@pytest.mark.parametrize("kw,name", [
    (dict(temperature=[0.5, -1.0]), "temperature of prompt 1"), (dict(temperature=[math.nan, 0.5]), "temperature of prompt 0"),
    (dict(temperature=[0.5, 1e31]), "temperature of prompt 1"), (dict(temperature=math.inf, top_k=4), "temperature of prompt 0"),
    (dict(temperature=float(torch.tensor(1e30)), top_k=4), "temperature of prompt 0"),
    (dict(top_p=[0.9, -0.1]), "top_p of prompt 1"), (dict(top_p=[math.nan, 0.1]), "top_p of prompt 0"),
    (dict(min_p=1.5), "min_p of prompt 0"), (dict(min_p=[0.0, -0.5]), "min_p of prompt 1"),
    (dict(min_p=[0.5, math.nan]), "min_p of prompt 1")])
def test_bad_values_are_refused_before_the_first_forward(run, monkeypatch, kw, name):
    monkeypatch.setattr(T._Model, "prefill", lambda *a, **k: pytest.fail("a forward ran"))
    with pytest.raises(ValueError, match=name + " is out of range"):
        run(**kw)


@pytest.mark.parametrize("kw", [dict(top_p=[0.5, 7.0]), dict(top_p=[math.inf, 0.0]), dict(min_p=[0.0, 1.0]),
                                dict(temperature=[9e29, 0.0]), dict(top_k=[-3, 1000])])
def test_ends_of_the_ranges_are_taken(run, kw):
    assert run(**kw)[1] == {"rows"}


@pytest.mark.parametrize("uniforms", [torch.rand(1, 2), torch.rand(24, 5), torch.rand(3)])
def test_greedy_rows_read_no_uniforms(run, uniforms):
    """As the scalar path: at temperature 0 the tensor is not looked at, whatever its shape."""
    want, _ = run(temperature=0.0, uniforms=uniforms)
    for kw in (dict(temperature=[0.0, 0.0]), dict(temperature=0.0, top_k=5), dict(temperature=0.0, min_p=0.1)):
        assert run(uniforms=uniforms, **kw) == (want, {"rows"})
