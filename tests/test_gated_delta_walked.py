"""The binding leaves a workspace out exactly where the library walks, as the library says."""
from state_space_model_selective_gb300 import binding
from tests.test_heads_boundary import ALIGN, L, P, WS, delta  # noqa: F401


def test_walked_sequences_need_no_workspace(L):  # noqa: F811
    steps = binding.ssm_gated_delta_walked_steps()
    assert 1 <= steps < 64
    bad = P(11, 8)  # refused for its address, after the workspace has been looked at
    for n in (1, steps):
        assert delta(L, n=n, kept=None, ws=None, nw=0, q=bad) == ALIGN
        assert delta(L, n=n, ws=None, nw=0, q=bad) == WS  # (what is kept is made in chunks)
    assert delta(L, n=steps + 1, kept=None, ws=None, nw=0, q=bad) == WS
    for n in (steps + 1, 5000):  # fp32 is walked at any length
        assert delta(L, n=n, it=0, kept=None, ws=None, nw=0, q=bad) == ALIGN
