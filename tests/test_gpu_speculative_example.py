"""The speculative decoding example: drafts change the number of steps, never the tokens (greedy decoding)."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_drafts_do_not_change_greedy_tokens():
    from mamba2_ssd_varlen_gb300 import build
    build.build()
    import speculative_s6
    same, agree, other = speculative_s6.main(new_tokens=24)
    assert same
    assert agree > 3.5  # the same model drafts: every draft is accepted but where the last step is cut
    assert 1.0 <= other < agree


def test_sampling_runs_and_accepts_some():
    import speculative_s6 as s
    import torch
    prompts = [torch.randint(64, (20 + i,)).tolist() for i in range(3)]
    target, draft = s.S6Model(64, 64, 2, 18, seed=0), s.S6Model(64, 64, 2, 18, seed=0)
    out, rate = s.generate(target, draft, prompts, 12, 2, temperature=1.0)
    assert all(len(o) >= 12 and all(0 <= t < 64 for t in o) for o in out) and rate > 2.0
