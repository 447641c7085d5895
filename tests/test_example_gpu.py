"""examples/kv4_decode.py runs the 4-bit operators together over several steps with growing caches."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "kv4_decode.py")


def load():
    spec = importlib.util.spec_from_file_location("kv4_decode", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("batch,heads,drafts,prompt,page", [(3, 8, 4, 100, 16), (5, 16, 9, 700, 64), (2, 5, 1, 40, 1)])
def test_steps(batch, heads, drafts, prompt, page):
    """O against float64 over the rows read back (their RoPE part rounded to bf16: 2^-9 of a key, as O itself)."""
    mod = load()
    error, _, dec = mod.main(batch, heads, drafts, prompt, 5, page, seed=batch)
    assert error < 2.0 ** -7
    held = sum(len(x) for x in dec.table_host)
    assert held == sum(-(-n // page) for n in dec.seq_lens.tolist())
    every = [p for x in dec.table_host for p in x] + dec.free_host
    assert sorted(every) == list(range(dec.pool.shape[0] // page))  # no page lost or held twice
