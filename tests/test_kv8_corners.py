"""Corners of the paged cache in 8 bits (KVCache over float8_e4m3fn blocks), against plain forms in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

from test_kv import TYPES  # noqa: E402
from test_kv8 import case8, check8  # noqa: E402
from test_kv_ranges import tk  # noqa: E402,F401


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,most", [(4, 4), (8, 2), (2, 8), (5, 3)])
def test_ragged_units_of_up_to_16_rows(tk, dtype, d, group, most):
    """Units of 1 to 8 rows and of 9 to 16 one after the other in every worker: a piece is not asked for its rows any more
    when the next ones may be in its place."""
    gen = torch.Generator().manual_seed(10 * group + d)
    new = torch.randint(0, most + 1, (420,), generator=gen).tolist()
    new[0] = most
    ctx = torch.randint(0, 40, (420,), generator=gen).tolist()
    q, eight, k, v, off, lens, table = case8(gen, new, ctx, 2 * group, 2, d, 16, dtype)
    got = check8(tk, q, eight, k, v, off, lens, table, max_new=most)
    c = [x.cuda() for x in eight]
    cache, ws, args = tk.KVCache(*c, dtype), tk.KVWorkspace(), [x.cuda() for x in (q, off, lens, table)]
    for _ in range(50):
        assert torch.equal(cache.attend(*args, ws, max_new=most), got)
    ws.status()
