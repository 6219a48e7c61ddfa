"""Outputs and workspaces of the decoder-step operators that overlap one another or an input are refused, on the host
(fake pointers that are never dereferenced)."""
import pytest

from tests.test_step_abi import FAKE, FAR, batch, cache, calls, logits


@pytest.fixture(scope="module")
def bi():
    import __graft_entry__
    __graft_entry__.build()
    import invariant_quantized_linear_gb300 as m
    return m


def test_logits_results_and_workspace_overlap_nothing(bi):
    """4 rows of 1000: logits at FAKE (8000 bytes), out at FAR (16000), argmax at 2 FAR (16), the workspace at 3 FAR."""
    n = bi.bi_logits_workspace_size(4)
    last = 7999 // 16 * 16
    for o in ({"am": FAKE}, {"am": FAKE + last}, {"am": FAR}, {"am": FAR + 15996}, {"am": FAR - 12}, {"am": 3 * FAR + n - 4},
              {"ws": FAKE}, {"ws": FAKE + last}, {"ws": FAR + 15984}, {"ws": FAR - n + 16}, {"ws": 2 * FAR}, {"out": FAKE + 7996}):
        assert logits(bi, **o) == bi.BI_ERR_INVALID_ARG, o
    # without one of the results, the other is still looked at
    assert logits(bi, out=None, am=FAKE + 4) == bi.BI_ERR_INVALID_ARG
    assert logits(bi, out=None, ws=2 * FAR) == bi.BI_ERR_INVALID_ARG
    assert logits(bi, am=None, ws=FAR) == bi.BI_ERR_INVALID_ARG


def test_logits_results_and_workspace_overlap_no_rule(bi):
    rows, R = 16, 5 * FAR
    history = dict(ids=6 * FAR, begin=R, mid=R + rows, end=R + 2 * rows)
    for r, o in ((history, {"am": R}), (history, {"am": R + rows + 12}), (history, {"out": R + 2 * rows}), (history, {"ws": R}),
                 ({"repetition": R}, {"am": R + 8}), ({"presence": R}, {"out": R - 4}), ({"frequency": R}, {"ws": R}),
                 ({"bias_ids": R, "bias": R + 1024, "n_bias": 7}, {"am": R + 108}),
                 ({"bias_ids": R, "bias": R + 1024, "n_bias": 7}, {"out": R + 1024}),
                 ({"mask": R, "ld_mask": 40}, {"am": R + 3 * 160 + 124}), ({"mask": R, "ld_mask": 40}, {"ws": R + 16}),
                 ({"mask": R, "ld_mask": 40}, {"out": R + 4})):
        assert logits(bi, r, **o) == bi.BI_ERR_INVALID_ARG, (r, o)


def test_attention_workspace_overlaps_nothing(bi):
    """6 rows of 8 heads of 128: q at FAR (rows of 1024), o at 2 FAR."""
    f = calls(bi)["attention"]
    need = bi.bi_attention_kv4_workspace_size(8, cache(bi), batch(bi))
    assert need > 16384
    for ws in (FAR, FAR + 12272, FAR - need + 16, 2 * FAR, 2 * FAR + 12272, 2 * FAR - need + 16):
        assert f(cache(bi), batch(bi), ws=ws) == bi.BI_ERR_INVALID_ARG, hex(ws)
