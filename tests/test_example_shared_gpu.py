"""examples/shared_decode.py: samples of shared prompts over several steps, with forks and releases between them."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "shared_decode.py")


def load():
    spec = importlib.util.spec_from_file_location("shared_decode", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("prompts,samples,heads,drafts,page,layers", [((300, 0, 129), 5, 8, 4, 4, 2), ((700,), 9, 16, 6, 1, 1),
                                                                      ((64, 1), 3, 5, 9, 64, 3)])
def test_steps(prompts, samples, heads, drafts, page, layers):
    """O against float64 (its own rounding and that of the weights: 2^-9 each of a key's size), the rows that every
    request holds bit for bit, every page's count."""
    mod = load()
    error, _, dec, own, grown = mod.main(prompts, samples, heads, drafts, 500, 7, page, layers, seed=samples)
    assert error < 2.0 ** -7 and grown > 7 * len(prompts)
    refs = torch.zeros_like(dec.refs)
    for b, x in enumerate(own):
        assert torch.equal(mod.held_rows(dec, b), x)
        n = -(-x.shape[1] // page)
        refs += torch.bincount(dec.table[b, :n].long(), minlength=refs.numel()).to(torch.int32)
    assert torch.equal(refs, dec.refs)
    assert int((refs > 1).sum()) > 0 or page == 64  # pages are shared
