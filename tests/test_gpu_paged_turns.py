"""Attention over a paged cache where a piece of a sequence is several units long: a wave then takes
several turns, with a running maximum, the pages looked up a turn ahead and its tile of values
overwritten; and more pieces than a wave joins at once."""
import pytest
import torch

import layer_ref
import mixer_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
UNIT = 128                 # tokens that a piece is a multiple of


def cache(seed, lens, P, Hk, D, dt):
    """(k, v, table) with the pages of `lens` tokens in random order on the GPU, NaN in unused slots."""
    r = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // P) for n in lens]
    order = torch.randperm(sum(need) + 2, generator=r, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    kv = [torch.randn(sum(need) + 2, P, Hk, D, generator=r, device="cuda").to(DT[dt]) for _ in range(2)]
    at = 0
    for n, (L, c) in enumerate(zip(lens, need)):
        table[n, :c] = order[at:at + c]
        for t in kv:
            t[order[at + c - 1].item(), L - (c - 1) * P:] = float("nan")
        at += c
    for t in kv:
        t[order[at:].long()] = float("nan")
    return (*kv, table)


def pieces(lens, window, Hk, P):
    """(units of a piece, pieces of each sequence) that the kernel cuts these lengths into: about 2048 workgroups."""
    lo = [max(0, n - window) if window else 0 for n in lens]
    units = [-(-(n - a // 32 * 32) // UNIT) for n, a in zip(lens, lo)]
    row = -(-max(lens) // P) * P
    share = min(max(1, 2048 // Hk), len(lens) * (-(-(min(row, window) if window else row) // UNIT) + 1))
    per = max(1, -(-sum(units) // share))
    return per, [max(1, -(-u // per)) for u in units]


def compare(gdn, q, k, v, table, lens, window, heads):
    n = torch.tensor(lens, device="cuda")
    o = gdn.paged_attn(q, k, v, table, n, window=window)
    torch.cuda.synchronize()
    at = torch.tensor(heads, device="cuda")
    want, err = ref.attn(q[:, at], k[:, :, at], v[:, :, at], table, n, None, window)
    layer_ref.check(o[:, at], want, err, "o")


# the window starts and ends inside pieces
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 2500])
@pytest.mark.parametrize("Hk,D,P", [(128, 64, 16), (128, 128, 24), (128, 256, 7), (64, 200, 64)])
def test_pieces_of_several_units(gpu_lib, dt, window, Hk, D, P):
    lens = (3000, 700, 4097, 1)
    per, cut = pieces(lens, window, Hk, P)
    assert per >= (3 if Hk == 128 else 2) and max(cut) > 1
    k, v, table = cache(1, lens, P, Hk, D, dt)
    r = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(4, Hk, D, generator=r, device="cuda").to(DT[dt])
    compare(gpu_lib, q, k, v, table, lens, window, (0, Hk // 2 + 1, Hk - 1))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,P", [(64, 16), (256, 24)])
def test_maximum_in_a_later_turn(gpu_lib, dt, D, P):
    """Keys that grow along the sequence: every turn replaces the maximum, the last one by far; and that shrink."""
    lens, Hk = (4097, 1000), 128
    assert pieces(lens, 0, Hk, P)[0] >= 3
    k, v, table = cache(3, lens, P, Hk, D, dt)
    r = torch.Generator(device="cuda").manual_seed(4)
    q = torch.rand(2, Hk, D, generator=r, device="cuda").to(DT[dt])
    for n, L in enumerate(lens):
        t = torch.arange(L, device="cuda")
        grow = (t / L * 30 if n == 0 else (L - t) / L * 30)[:, None, None] * D ** -0.5
        page, slot = table[n, t // P].long(), t % P
        k[page, slot] = (k[page, slot].float().abs() * grow).to(k.dtype)
    compare(gpu_lib, q, k, v, table, lens, 0, (0, 127))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 256])
def test_absent_pages_in_a_later_turn(gpu_lib, dt, D, monkeypatch):
    """Pages that are not there, in turns after a piece's first: single ones, a whole turn, a whole piece."""
    lens, Hk, P = (4000, 2000), 128, 16
    per, _ = pieces(lens, 0, Hk, P)
    assert per >= 3
    k, v, table = cache(5, lens, P, Hk, D, dt)
    table[0, 10], table[0, 17:26], table[1, 100:] = -1, k.shape[0], -7       # 16 tokens each
    table[0, 8 * per:16 * per] = -1                                          # the second piece
    r = torch.Generator(device="cuda").manual_seed(6)
    q = torch.randn(2, Hk, D, generator=r, device="cuda").to(DT[dt])
    monkeypatch.setenv("GDN_DEBUG", "0")                                     # (which would refuse them)
    compare(gpu_lib, q, k, v, table, lens, 0, (1, 126))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_more_pieces_than_a_wave(gpu_lib, dt):
    """One sequence of 80 pieces, its largest score in the last one."""
    lens, P = (10200,), 64
    per, cut = pieces(lens, 0, 1, P)
    assert per == 1 and cut[0] > 64
    k, v, table = cache(7, lens, P, 1, 64, dt)
    r = torch.Generator(device="cuda").manual_seed(8)
    q = torch.rand(1, 1, 64, generator=r, device="cuda").to(DT[dt])
    k[table[0, 159].long(), 10] = 1.0
    compare(gpu_lib, q, k, v, table, lens, 0, (0,))
