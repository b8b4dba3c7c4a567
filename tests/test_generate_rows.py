"""Generation with top-k, min-p and parameters per prompt: the driver's part on
the CPU with stand-ins, and the kernels' picks on the GPU against the 64-bit
definition of the row sampler."""
import pytest
import torch

import paged_reference as R
from workloads import TINY, make_tokens, make_uniforms, make_weights

llb = pytest.importorskip("decoder_only_transformer_llama_b200",
                          reason="library not built (run decoder_only_transformer_llama_b200/build.py)")
import decoder_only_transformer_llama_b200.generate as G  # noqa: E402


class _Model:
    """A stand-in whose logits depend on the last token and its position only."""

    class args:
        max_seq_len, vocab_size, max_batch_size = 24, 50, 3

    class arena:
        device = torch.device("cpu")

    def _row(self, tok, pos):
        return torch.randn(50, generator=torch.Generator().manual_seed(1000 * int(tok) + int(pos)))

    def prefill(self, tokens, logits=None, all_logits=False):
        for b in range(tokens.shape[0]):
            logits[b].copy_(self._row(tokens[b, -1], tokens.shape[1] - 1))

    def decode_step(self, tokens, pos, logits=None):
        for b in range(tokens.shape[0]):
            logits[b].copy_(self._row(tokens[b], pos[b]))

    def status(self):
        return 0


def _rows(logits, temperature, uniforms, out, top_k=None, top_p=None, min_p=None, stream=None):
    for b in range(logits.shape[0]):
        out[b] = R.sample(logits[b], float(temperature[b]), int(top_k[b]), float(top_p[b]), float(min_p[b]),
                          float(uniforms[b]))
    return out


def test_driver_passes_each_prompts_parameters(monkeypatch):
    m = _Model()
    monkeypatch.setattr(G, "sample_rows", _rows)
    monkeypatch.setattr(G, "sample", lambda *a, **k: pytest.fail("the scalar sampler was called"))
    u = torch.rand(24, 3, generator=torch.Generator().manual_seed(2))
    prompts = [[1, 2, 3], [4, 5], [6, 7, 8, 9]]
    t, k, p, mp = [0.9, 0.0, 1.4], [3, 0, 0], [1.0, 0.9, 0.7], [0.0, 0.0, 0.1]
    out, lp = G.generate(m, prompts, max_gen_len=6, temperature=t, top_p=p, top_k=k, min_p=mp, uniforms=u, echo=True)
    assert lp is None
    for b, seq in enumerate(out):
        assert seq[:len(prompts[b])] == prompts[b] and len(seq) == len(prompts[b]) + 6
        for pos in range(len(prompts[b]), len(seq)):
            want = R.sample(m._row(seq[pos - 1], pos - 1), float(torch.tensor(t[b])), k[b], float(torch.tensor(p[b])),
                            float(torch.tensor(mp[b])), float(u[pos, b]))
            assert seq[pos] == want
    one, _ = G.generate(m, prompts, max_gen_len=6, temperature=0.9, top_k=1, uniforms=u)
    greedy, _ = G.generate(m, prompts, max_gen_len=6, temperature=[0.0] * 3)
    assert one == greedy


def test_driver_refuses_bad_parameters(monkeypatch):
    m = _Model()
    monkeypatch.setattr(G, "sample_rows", _rows)
    u = torch.zeros(24, 2)
    for kw in (dict(temperature=[1.0]), dict(top_k=[1, 2, 3]), dict(min_p=[0.1]), dict(top_p=[0.9, 0.9, 0.9])):
        with pytest.raises(ValueError, match="entries"):
            G.generate(m, [[1], [2]], max_gen_len=2, uniforms=u, **kw)
    with pytest.raises(ValueError, match="out of range"):
        G.generate(m, [[1], [2]], max_gen_len=2, uniforms=u, min_p=[0.0, 1.5])
    with pytest.raises(ValueError, match="uniforms"):
        G.generate(m, [[1], [2]], max_gen_len=2, temperature=[0.0, 1.0])


@pytest.mark.gpu
def test_generation_with_rows_of_their_own(cuda_device, monkeypatch):
    from tests.helpers import build_model
    s = TINY
    m = build_model(s, make_weights(s, 71))
    toks = make_tokens(s.vocab_size, (2, 9), 72)
    prompts = [toks[0, :5].tolist(), toks[1, :9].tolist()]
    uni = make_uniforms((s.max_seq_len, 2), 73).cuda()
    seen = []

    def recorded(logits, temperature, uniforms, out, **kw):
        llb.sample_rows(logits, temperature, uniforms, out, **kw)
        seen.append((logits.cpu().clone(), uniforms.cpu().clone(), out.cpu().clone()))
        return out

    monkeypatch.setattr(G, "sample_rows", recorded)
    f = lambda x: float(torch.tensor(x, dtype=torch.float32))
    t, k, p, mp = [0.8, 1.2], [20, 0], [0.95, 0.9], [0.0, 0.05]
    out, _ = G.generate(m, prompts, max_gen_len=8, temperature=t, top_p=p, top_k=k, min_p=mp, uniforms=uni, echo=True)
    assert len(seen) == 9 + 8 - 5
    for logits, u, picked in seen:
        assert picked.tolist() == [R.sample(logits[b], f(t[b]), k[b], f(p[b]), f(mp[b]), float(u[b])) for b in range(2)]
    # position of step i: the shortest prompt's end plus i
    for b, seq in enumerate(out):
        for pos in range(len(prompts[b]), len(seq)):
            assert seq[pos] == int(seen[pos - 5][2][b])
    one, _ = G.generate(m, prompts, max_gen_len=8, temperature=0.7, top_k=1, uniforms=uni)
    greedy, _ = G.generate(m, prompts, max_gen_len=8, temperature=0.0)
    assert one == greedy
    m.close()
