"""How calls on the paged cache are dispatched, and streams."""
import pytest
import torch

from hybrid_linear_attention_packed_gb300 import spanla
from paged_helpers import E4M3, check_attention
from test_gpu_paged_attention import _run, _setup, weights

pytestmark = pytest.mark.gpu


def _launches(kernel):
    return spanla.profile_read()[kernel]["launches"]


@pytest.mark.parametrize("lens,rows,G,max_rows,expands", [
    ([700, 40, 520, 9], [260, 1, 270, 9], 8, 270, True),      # the caller names a sequence of 2,160 row heads
    ([700, 40, 520, 9], [260, 1, 270, 9], 8, None, False),    # 135 rows on average, which is all that the host knows
    ([700, 520], [260, 270], 8, None, True),
    ([300] * 256, [1] * 256, 8, None, False),                 # single tokens, of which the call does not say so
])
def test_when_quantised_pages_are_expanded(cuda_device, lens, rows, G, max_rows, expands):
    q, c, table, cu = _setup(lens, rows, G, 2, 16, E4M3, cuda_device, seed=41)
    before = _launches("kv_expand")
    out, lse = _run(q, c, table, lens, cu, cuda_device, max_rows=max_rows)
    assert _launches("kv_expand") - before == int(expands)
    check_attention(q, out, lse, c, table, lens, cu, 0.125, weights(G, E4M3))
