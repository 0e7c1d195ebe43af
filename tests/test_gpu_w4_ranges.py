"""The 4-bit weight and its layer, and the heads behind it, at the ends of the
ranges that the checks of arguments accept; the former bit for bit (w4_exact:
every sum is exact)."""
import numpy as np
import pytest
import torch

import lora_row_adapter_amd as lr
import w4_exact as E
import w4_ref as R
from gpu_helpers import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the gpu tests need an MI355X")
    torch.cuda.set_device(0)
    lr.load_library()
    yield
    torch.cuda.synchronize()


@pytest.fixture(autouse=True)
def _freed():
    yield
    torch.cuda.empty_cache()  # the buffers here are of many GiB


def room(gib):
    """Skips where other programs hold the card's memory."""
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0] >> 30
    if free < gib:
        pytest.skip("%d GiB free of the %d that this takes" % (free, gib))


def test_pages_past_32_bits():
    """Adapters in pages of 32 and of 64 GiB: places in them, counted in 16
    bytes, are shifted by 31 and by 32 bits."""
    room(70)
    k, ds, group, R = 264, (48, 40), 64, 16
    W = E.Weight(1, sum(ds), k, group)
    Wp = lr.lora_w4_pack(W.packed(), W.s, k, group, zeros=W.z)
    dense = W.dense()
    pool = torch.empty(1 << 36, dtype=torch.uint8, device="cuda")
    for page, ranks in ((1 << 35, [16, 8]), (1 << 36, [16])):
        S = len(ranks)
        sets = [E.adapters(10 + i, S, R, k, d, ranks) for i, d in enumerate(ds)]
        scales = [2.0, 0.5][:S]
        rk = torch.tensor(ranks, dtype=torch.int32).cuda()
        sc = torch.tensor(scales, dtype=F32).cuda()
        for M in (1, 9, 30, 50):
            say("w4 layer, pages of 2^%d bytes, %d rows" % (page.bit_length() - 1, M))
            ids = np.arange(M) % (S + 1) - (M > 1)
            ids_d = torch.from_numpy(ids.astype(np.int32)).cuda()
            x = E.rows(M, M, k)
            for n in range(len(ds)):  # one slice's adapters fill the pool at a time
                A, B = sets[n]
                table = torch.tensor([[S - 1 - i] for i in range(S)], dtype=torch.int32).cuda()
                for i, r in enumerate(ranks):
                    raw = torch.cat([A[i, :r].reshape(-1), B[i, :, :r].reshape(-1)]).view(torch.uint8)
                    at = (S - 1 - i) * page
                    pool[at:at + raw.numel()] = raw
                ad = [lr.Adapters.slots(a, b, rk) for a, b in sets]
                ad[n] = lr.Adapters.paged(pool, table, rk, page, R)
                y = lr.lora_linear_sliced_w4(x, Wp, [lr.Slice(d, a, sc) for d, a in zip(ds, ad)], ids_d)
                want, _ = E.layer(x, dense, ds, sets, ranks, scales, ids, twice=M > 32)
                assert torch.equal(y, want)


def bytes_at_random(seed, *shape):
    t = torch.empty(shape, dtype=torch.uint8, device="cuda")
    t.view(-1).view(torch.int64).random_(generator=torch.Generator(device="cuda").manual_seed(seed))
    return t


def test_pack_past_a_launch():
    """More records (2^24) than a launch has threads for: all as when 4096 rows
    are laid out at a time."""
    room(80)
    d, k, group, step = (1 << 18) + 16, 1 << 17, 128, 4096
    say("w4 pack, %d records" % (d // 16 * k // 128))
    q, z = bytes_at_random(1, d, k // 2), bytes_at_random(2, d, k // group)
    s = (bytes_at_random(3, d, k // group).to(BF) - 100) / 64
    W = lr.lora_w4_pack(q, s, k, group, zeros=z)
    for r in range(0, d, step):
        part = lr.lora_w4_pack(q[r:r + step], s[r:r + step], k, group, zeros=z[r:r + step])
        at = r // 16 * (k // 128) * 1088
        n = part.data.numel()
        assert torch.equal(W.data[at:at + n], part.data)
    last = lr.lora_w4_dequantize(part, F32)  # and by the definition
    codes = torch.stack([q[r:] & 15, q[r:] >> 4], -1).flatten(1)
    want = s[r:].float().repeat_interleave(group, 1) * (codes.float() - (z[r:] % 32).float().repeat_interleave(group, 1))
    assert torch.equal(last, want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_read_back_past_a_launch(dtype):
    """As many rows as take 2^24 workgroups and three more."""
    room(60)
    d, k, step = (1 << 28) + 48, 8, 1 << 24
    say("w4 read back, %d rows, %s" % (d, dtype))
    q = bytes_at_random(4, d, k // 2)
    s = (bytes_at_random(5, d, 1).to(BF) - 100) / 64
    W = lr.lora_w4_pack(q, s, k, 128)
    y = lr.lora_w4_dequantize(W, dtype)
    for r in range(0, d, step):
        codes = torch.stack([q[r:r + step] & 15, q[r:r + step] >> 4], -1).flatten(1)
        want = (s[r:r + step].float() * (codes.float() - 8)).to(dtype)  # 8 by 4 bits: exact in fp32
        assert torch.equal(y[r:r + step], want)


def test_heads_past_a_launch():
    """As many heads, of a size that a workgroup takes four of, as take 2^24
    workgroups and two more; in place.  Tolerance as in the heads' own tests."""
    room(130)
    M, D, eps = (1 << 26) + 7, 912, 1e-6
    say("heads, %d rows of %d" % (M, D))
    q = torch.empty(M, 1, D, dtype=BF, device="cuda")
    pos = torch.full((M,), -1, dtype=torch.int64, device="cuda")
    at = torch.tensor([0, 5, (1 << 24) - 1, 1 << 24, (1 << 25) - 1, 1 << 25, (1 << 25) + 1, (1 << 26) - 1, 1 << 26, M - 1])
    g = torch.Generator().manual_seed(6)
    x = torch.randn(len(at), 1, D, generator=g).to(BF)
    beside = at[:-1] + 1  # padding rows, left as they are
    beside = beside[~torch.isin(beside, at)]
    pad = torch.randn(len(beside), 1, D, generator=g).to(BF)
    q[at.cuda()], q[beside.cuda()] = x.cuda(), pad.cuda()
    p = torch.randint(0, 100000, (len(at),), generator=g)
    pos[at.cuda()] = p.cuda()
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(BF)
    inv = torch.tensor([1e4 ** (-2 * i / D) for i in range(D // 2)], dtype=F32)
    lr.lora_qk_norm_rope(q, None, pos, lr.Rope(inv.cuda()), w.cuda(), eps=eps, q_out=q)
    angle = p.double().numpy()[:, None] * inv.double().numpy()
    want, mag = R.heads(x.double().numpy(), w.double().numpy(), eps, np.cos(angle), np.sin(angle), D, False)
    got = q[at.cuda()].cpu().double().numpy()
    assert (np.abs(got - want) <= 2.0 ** -21 * mag + 2.0 ** -8 * np.abs(want)).all()
    assert torch.equal(q[beside.cuda()].cpu(), pad)
