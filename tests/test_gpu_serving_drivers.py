"""The serving drivers where calls meet: side streams, refused calls, idle rows, layers
without a window, states that are taken up again."""
import numpy as np
import pytest
import torch

from oracle import serving

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods(cuda_ok):
    from long_context_compressed_compress_b200 import build
    build.build()
    from long_context_compressed_compress_b200 import layer, ops, paged
    return layer, ops, paged


def np64(t):
    return t.detach().cpu().double().numpy()


def test_host_lists_on_a_busy_side_stream(mods):
    """The current stream takes and fills memory of the lists' size while the side stream
    has yet to read them."""
    _, _, paged = mods
    c = paged.PagedEntries(1, 64, 4, 8, 12, 60)
    m = serving.Pages(64, 4, 12, c.max_pages, c.pool.float().cpu().numpy())
    a = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    keep = []
    for name, args in (("reserve", ([0, 3], [17, 8])), ("fork", ([0, 0, 3], [1, 2, 4], [17, 16, 5])), ("free", ([0, 2],)),
                       ("reserve", ([0, 1], [30, 40]))):
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for _ in range(20):                        # some milliseconds
                a = (a @ a).clamp(-1, 1)
        getattr(c, name)(*args, stream=s)
        getattr(m, name)(*args)
        keep += [torch.full((k,), 10 ** 9, dtype=torch.int32, device="cuda") for k in (1, 2, 3, 4) for _ in range(8)]
        torch.cuda.synchronize()
        assert c.status.item() == 0
        np.testing.assert_array_equal(c.held.cpu().numpy(), [len(r) for r in m.rows])
        np.testing.assert_array_equal(c.table.cpu().numpy(), m.table())
        np.testing.assert_array_equal(c.refcount.cpu().numpy(), m.ref)
