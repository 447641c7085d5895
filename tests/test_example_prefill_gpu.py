"""examples/kv4_decode.py: prompts that are empty, replace another one, or do not fit."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_example_gpu import load  # noqa: E402


def prompt(n):
    return torch.randn((n, 576), device="cuda").to(torch.bfloat16)


def test_no_page_is_lost():
    dec = load().Kv4Decoder(2, 2, 3, 100, 12, 16)
    every = list(range(12))
    held = lambda: sorted(dec.free_host + dec.table_host[0] + dec.table_host[1])  # noqa: E731
    for b, n in ((0, 0), (1, 40), (0, 96), (1, 17), (1, 0), (0, 1), (1, 100)):
        x = prompt(n)
        dec.prefill(b, x[:, :512], x[:, 512:])
        assert int(dec.seq_lens[b]) == n and len(dec.table_host[b]) == -(-n // 16)
        assert dec.table[b, :len(dec.table_host[b])].tolist() == dec.table_host[b]
        assert held() == every
    assert dec.v.status() == 0


@pytest.mark.parametrize("pages,n", [(3, 49), (12, 113)])
def test_a_prompt_that_does_not_fit_is_refused(pages, n):
    """More pages than are free; more than the table's columns."""
    dec = load().Kv4Decoder(2, 2, 3, 100, pages, 16)
    x = prompt(n)
    with pytest.raises(ValueError):
        dec.prefill(0, x[:, :512], x[:, 512:])
    assert sorted(dec.free_host) == list(range(pages)) and not dec.table_host[0]
    assert int(dec.seq_lens[0]) == 0


def test_a_request_without_a_prompt_decodes():
    mod = load()
    dec = mod.Kv4Decoder(1, 2, 2, 40, 8, 8)
    e = prompt(0)
    dec.prefill(0, e[:, :512], e[:, 512:])
    dec.new_lens.fill_(2)
    dec.parents.copy_(torch.tensor([-1, 0], dtype=torch.int32))
    for x in (dec.tokens, dec.q_nope, dec.q_rope):
        x.normal_()
    o, _ = dec.step()
    ref = mod.exact(dec, 0, 0, 2)
    assert float((o[:2].double() - ref).norm() / ref.norm()) < 2.0 ** -7
    dec.accept([[0, 1]])
    assert dec.seq_lens.tolist() == [2] and np.array_equal(len(dec.table_host[0]), 1)
