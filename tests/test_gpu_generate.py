"""The decoder-step operators run together as a decoder runs them: generation
with and without drafts gives the same tokens, and a prompt in one pass the
same logits as the prompt a token at a time."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import step_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gen():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "generate.py")
    spec = importlib.util.spec_from_file_location("example_generate", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def small(gen, **o):
    return gen.Config(**{**dict(layers=2, hidden=256, heads=4, kv_heads=2, head_size=64, inner=384, vocab=1003, page=16,
                                max_len=256), **o})


def prompts(cfg, lengths, seed=3):
    rng = np.random.default_rng(seed)
    return [rng.integers(0, cfg.vocab, n).tolist() for n in lengths]


@pytest.mark.parametrize("rules", [{}, dict(repetition=1.3, presence=0.25, frequency=0.125), "mask"])
@pytest.mark.parametrize("o", [{}, dict(head_size=128, heads=8, page=32)])
def test_drafts_change_nothing(gen, o, rules):
    cfg = small(gen, **o)
    ps = prompts(cfg, (2, 37, 16))
    if rules == "mask":                                    # few allowed tokens: texts repeat, drafts are accepted
        words = np.zeros((1, (cfg.vocab + 31) // 32), np.uint32)
        for i in (5, 77, 1002):
            words[0, i >> 5] |= np.uint32(1 << (i & 31))
        rules = dict(mask=torch.from_numpy(words.view(np.int32)).cuda())
    plain, p0 = gen.generate(gen.Decoder(cfg, 3), ps, 40, 0, **rules)
    model = gen.Decoder(cfg, 3)
    spec, p1 = gen.generate(model, ps, 40, 5, **rules)
    assert plain == spec and all(len(t) == len(p) + 40 for t, p in zip(plain, ps))
    assert p0 == 40 and p1 <= p0
    if "mask" in rules:
        assert p1 < p0 and all(t in (5, 77, 1002) for s, p in zip(spec, ps) for t in s[len(p):])
    assert gen.bi.bi_workspace_status(model.attn_ws) == gen.bi.BI_OK


def test_prompt_at_once_and_token_by_token(gen):
    cfg = small(gen)
    text = prompts(cfg, (33,))[0]
    ids = torch.tensor(text, dtype=torch.int32, device="cuda")
    one = gen.Decoder(cfg, 1).forward(ids, [33], [33], torch.arange(33, device="cuda"))
    model = gen.Decoder(cfg, 1)
    row = torch.zeros(1, dtype=torch.long, device="cuda")
    for i in range(33):
        assert torch.equal(model.forward(ids[i:i + 1], [1], [i + 1], row)[0], one[i]), i
