"""Generation from a decoder whose MLPs are experts in e4m3: drafts change nothing, and a prompt in one pass has the logits
of the prompt a token at a time."""
import numpy as np
import pytest
import torch

from tests.test_gpu_generate import gen, prompts, small  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("o", [dict(experts=5), dict(experts=9, top_k=3, inner=272)])
def test_drafts_change_nothing(gen, o):  # noqa: F811
    cfg = small(gen, **o)
    ps = prompts(cfg, (2, 37, 16))
    plain, steps = gen.generate(gen.Decoder(cfg, 3), ps, 20)
    model = gen.Decoder(cfg, 3)
    spec, passes = gen.generate(model, ps, 20, 4)
    assert plain == spec and passes <= steps
    assert gen.bi.bi_workspace_status(model.f8_ws) == gen.bi.BI_OK


def test_a_prompt_has_the_same_logits_in_any_parts(gen):  # noqa: F811
    cfg = small(gen, experts=6)
    prompt = np.random.default_rng(5).integers(0, cfg.vocab, 150).astype(np.int32)
    ids = torch.from_numpy(prompt).cuda()

    def run(cuts):
        model, logits, at = gen.Decoder(cfg, 1), [], 0
        for n in cuts:
            logits.append(model.forward(ids[at:at + n], [n], [at + n], torch.arange(n, device="cuda")))
            at += n
        return torch.cat(logits).view(torch.int16)
    whole = run([150])
    for cuts in ([1] * 5 + [145], [70, 1, 79], [149, 1]):
        assert torch.equal(run(cuts), whole), cuts
