"""Attention over the 8-bit paged cache where sizes lie far apart: pages, the step's own rows, rows of q.

The bounds are those of the attention tests: each score's error follows from that key's own products, the probabilities
are rounded once, and what a row does not see, or sees with a weight of 2^-60, has no part in its result."""

import numpy as np
import pytest
import torch

from test_gpu_kv8 import attention_case, check_attention, i32, reference, run_attention

pytestmark = pytest.mark.gpu


def set_exps(c, plane, table):
    """Exponent bytes of each sequence's pages, in the order of its tokens."""
    for b, s in enumerate(c["ids"]):
        for j in range(-(-int(c["lengths"][s]) // c["page"])):
            c["exps"][plane, c["tables"][s, j]] = table(b, j)
    c["cache"].exps[0] = torch.from_numpy(c["exps"])


@pytest.mark.parametrize("high", [150, 190, 247])
@pytest.mark.parametrize("order", ["small first", "large first", "in turn"])
@pytest.mark.parametrize("prefixes,nodes,hq,page,dtype", [
    ([200, 77], [1, 1], 4, 16, "bf16"), ([3000], [1], 4, 64, "bf16"), ([900, 130], [3, 2], 4, 32, "bf16"),
    ([300, 190], [30, 100], 4, 64, "bf16"), ([3000], [40], 8, 64, "bf16"), ([500], [17], 2, 128, "bf16")])
def test_weights_of_pages_whose_values_are_of_unlike_size(prefixes, nodes, hq, page, dtype, order, high):
    """V pages at the least scale (all zeros have it) beside very large ones: the weights do not depend on V."""
    c = attention_case(31, prefixes, nodes, hq, 1, page, dtype)
    blocks = [-(-p // page) for p in prefixes]
    # (in turn: no two scales within 64 keys)
    large = {"small first": lambda b, j: 2 * j >= blocks[b], "large first": lambda b, j: 2 * j < blocks[b],
             "in turn": lambda b, j: j * page // 64 % 2 == 1}[order]
    if page < 64:  # whole units of 64 keys
        was = large
        large = lambda b, j: was(b, j // (64 // page) * (64 // page))  # noqa: E731
    set_exps(c, 1, lambda b, j: high if large(b, j) else 67)
    # (448 * 2^120 is above the largest bf16, 1.99 * 2^127: an average above it is an infinity in bf16)
    (out, lse), ref = run_attention(c), reference(c)
    over = np.abs(ref[0]) > torch.finfo(out.dtype).max
    at = torch.from_numpy(over).cuda()
    assert np.array_equal(out[at].double().cpu().numpy(), np.sign(ref[0][over]) * np.inf)
    out[at], ref[0][over] = 0, 0
    check_attention(c, (out, lse), ref)
