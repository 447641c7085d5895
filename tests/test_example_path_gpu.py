"""examples/kv4_decode.py keeps the accepted path of a draft tree, whichever nodes it is made of."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from oracle import kv4  # noqa: E402
from test_example_gpu import load  # noqa: E402


def cached(dec, b):
    """The 4-bit rows of request b's cached tokens, in order."""
    pos = np.arange(int(dec.seq_lens[b]))
    pages = np.asarray(dec.table_host[b], np.int64)
    assert dec.table[b, :len(pages)].tolist() == list(pages)  # what the next step's kernels read
    return dec.pool.cpu().numpy()[pages[pos // dec.page] * dec.page + pos % dec.page]


def coded(x):
    h = x.float().cpu().numpy().astype(np.float64)
    if not len(h):
        return np.zeros((0, kv4.ROW_BYTES), np.uint8)
    return kv4.encode_rows(h[:, :512], h[:, 512:])


@pytest.mark.parametrize("page", [1, 4, 64])
def test_rows_of_the_accepted_paths(page):
    mod = load()
    dec = mod.Kv4Decoder(4, 2, 6, 200, 4 * (200 // page + 2), page)
    prompts = [torch.randn((n, 576), device="cuda").to(torch.bfloat16) for n in (1, 63, 64, 30)]
    for b, x in enumerate(prompts):
        dec.prefill(b, x[:, :512], x[:, 512:])
    held = [coded(x) for x in prompts]
    steps = [
        # parents, accepted path
        [([-1, 0, 0, 1, 2, 4], [0, 2, 4, 5]), ([-1, -1, 1, 2], [1, 2, 3]), ([-1, 0], []), ([-1, -1, -1], [2])],
        [([-1, 0, 1, 2, 3, 4], [0, 1, 2, 3, 4, 5]), ([], []), ([-1, 0, 0, 2], [0, 2, 3]), ([-1, 0, 1], [0])],
        [([-1], [0]), ([-1, -1, 0, 1, 3, 2], [1, 3, 4]), ([-1, -1], [1]), ([-1, 0, 0, 0, 0, 0], [0, 5])],
    ]
    for step in steps:
        new = [len(p) for p, _ in step]
        dec.new_lens.copy_(torch.tensor(new, dtype=torch.int32))
        dec.parents[:sum(new)] = torch.tensor([i for p, _ in step for i in p], dtype=torch.int32, device="cuda")
        dec.tokens.copy_(torch.randn(dec.tokens.shape, device="cuda").to(torch.bfloat16))
        dec.q_nope.normal_()
        dec.q_rope.normal_()
        dec.step()
        at = np.concatenate([[0], np.cumsum(new)])
        for b, (_, path) in enumerate(step):
            held[b] = np.concatenate([held[b], coded(dec.tokens[[int(at[b]) + i for i in path]])])
        dec.accept([path for _, path in step])
        for b in range(4):
            assert int(dec.seq_lens[b]) == len(held[b])
            assert np.array_equal(cached(dec, b), held[b])


def test_random_paths_are_paths():
    mod = load()
    rng = np.random.default_rng(0)
    for _ in range(200):
        n = int(rng.integers(0, 9))
        parents = np.array([int(rng.integers(-1, i)) if i else -1 for i in range(n)])
        path = mod.random_path(parents, rng)
        assert all(0 <= i < n for i in path)
        assert [-1] + path[:-1] == [int(parents[i]) for i in path] or not path
