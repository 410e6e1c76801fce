"""The hybrid example with one drawn row a prompt: a temperature that is given counts, whatever the number of samples."""
import pytest
import torch

from speculative_decode_gated_gdn_gb300 import lib as L
from tests.test_hybrid_example_gpu import load_example
from tests.test_sampled_example_gpu import check_attention, check_pages

pytestmark = pytest.mark.gpu


def test_one_drawn_row_a_prompt(gdn):
    run = load_example().run
    torch.manual_seed(0)
    m, _ = run(rows=4, prompt=40, cycles=9, draft=1, samples=1, temperature=3.0)
    assert m.B == 4 and m.refs is not None and (m.ways["temperature"] == 3.0).all()
    offsets = m.offsets
    assert (offsets >= 40 + 10).all() and (offsets <= 40 + 20).all()
    assert max(check_pages(m)) == 1  # nothing is shared
    check_attention(m)
    greedy, _ = run(rows=4, prompt=40, cycles=9, draft=1)
    assert greedy.refs is None
    # at this temperature over 512 tokens the rows go other ways than the most likely tokens do
    assert not torch.equal(m.tokens, greedy.tokens)
    cold, _ = run(rows=4, prompt=40, cycles=9, draft=1, samples=1, temperature=0.0)  # the first of the order: greedy's tokens
    assert torch.equal(cold.tokens, greedy.tokens) and torch.equal(cold.offsets, greedy.offsets)
    m.end(torch.arange(4, device="cuda"))
    assert m.compact() == 0 and L.gdn_get_status() == 0
