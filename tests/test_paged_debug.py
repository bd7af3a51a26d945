"""What GDN_DEBUG lets the paged cache's calls refuse: positions that a call uses, and no others (CPU; the
calls themselves on the GPU)."""
import pytest
import torch

from gated_delta_rule_14_amd import _mixer

P, POOL = 16, 20
MAX = 2 ** 63 - 1


class Stream:
    """Nothing to wait for on the CPU."""
    def synchronize(self):
        pass


def look(table, lens, **kw):
    _mixer._look(torch.zeros(POOL, P, 1, 64), torch.tensor(table, dtype=torch.int32), torch.tensor(lens),
                 stream=Stream(), dev=torch.device("cpu"), **kw)


@pytest.fixture(autouse=True)
def debug(monkeypatch):
    monkeypatch.setenv("GDN_DEBUG", "1")


def test_pages_before_the_window_may_be_gone():
    """lens 100, window 30: positions 70 to 99, the pages 4 to 6."""
    table = [[-1, -1, 99, -7, 3, 4, 5, -1], [1, -1, -1, -1, -1, -1, -1, -1]]
    look(table, [100, 16], window=30)
    for window in (0, 100, 37):                     # 37: position 63, page 3
        with pytest.raises(ValueError, match="page_table"):
            look(table, [100, 16], window=window)
    with pytest.raises(ValueError, match="page_table"):
        look([[-1, -1, 99, -7, 3, 4, POOL, -1]], [100], window=30)
    look(table, [0, 0], window=1)


def test_pages_that_an_append_does_not_write_may_be_gone():
    """Tokens go to positions lens .. lens + T - 1, whatever the table says of those before."""
    table = [[-1, 5, -1], [-1, -1, 2]]
    look(table, [16, 32], T=16)
    look(table, [17, 40], cu_seqlens=torch.tensor([0, 15, 23]), T=23)
    look(table, [3, 48], cu_seqlens=torch.tensor([0, 0, 0]), T=0)       # nothing to write
    for lens in ([15, 32], [17, 32]):
        with pytest.raises(ValueError, match="page_table"):
            look(table, lens, T=16)


@pytest.mark.parametrize("n", [-1, 49, MAX, MAX - 3, -MAX])
def test_lengths_outside_the_table(n):
    for kw in (dict(T=4), dict(T=0), dict(window=0), dict(window=5), dict(cu_seqlens=torch.tensor([0, 4]), T=4)):
        with pytest.raises(ValueError, match="lens"):
            look([[0, 1, 2]], [n], **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [1, 30, 200])
def test_calls_over_freed_pages(gpu_lib, window):
    """A cache whose pages before the window are given away: attention and append as over the whole one."""
    gdn, r = gpu_lib, torch.Generator().manual_seed(1)
    kc, vc = (torch.randn(POOL, P, 2, 64, generator=r).cuda() for _ in range(2))
    q, x = torch.randn(2, 4, 64, generator=r).cuda(), torch.randn(2, 3, 2, 64, generator=r).cuda()
    table = torch.randperm(POOL, generator=r)[:20].view(2, 10).to(torch.int32).cuda()
    lens = torch.tensor([150, 61]).cuda()
    want = gdn.paged_attn(q, kc, vc, table, lens, window=window)
    freed = table.clone()
    for n, L in enumerate(lens.tolist()):
        freed[n, :max(0, L - window) // P] = -1
        freed[n, -(-(L + 3) // P):] = -1
    assert torch.equal(gdn.paged_attn(q, kc, vc, freed, lens, window=window), want)
    if window == 200:
        return
    both = [(kc.clone(), vc.clone()) for _ in range(2)]
    gdn.paged_append(None, x, -x, *both[0], table, lens)
    gdn.paged_append(None, x, -x, *both[1], freed, lens)
    assert all(torch.equal(a, b) for a, b in zip(*both))
