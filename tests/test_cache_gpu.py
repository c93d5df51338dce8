"""The cache's writers and readers on the GPU against the oracle.

Tolerances.  A rotated value a cos - b sin is computed in float32 from exact bf16 inputs:
the angle is off by at most 2^-22 turns at |position| < 2^31 (the frequency's 2^-53 times
the position) plus 2^-25 turns of the float angle, i.e. 1.7e-6 rad, sine and cosine by
another 2e-7 and the three float32 roundings by 2^-24 each, so by at most 3e-6 (|a| + |b|)
in all; the one rounding to bf16 adds half a step, 2^-8 of the value.  Everything else is
copied or is exact arithmetic (IEEE float32 division, one rounding to E4M3), and has to be equal.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import cache_oracle as co
from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu

FREQ = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)


def _bf16(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def _rope_close(got, x, positions, sections, interleaved, freq=FREQ):
    """got, x: [T, H, 64] bf16 CPU tensors."""
    x = x.float().numpy()
    ref = co.rope(x, positions, freq, sections, interleaved)
    if interleaved:
        size = np.repeat(np.abs(x[..., 0::2]) + np.abs(x[..., 1::2]), 2, axis=-1)
    else:
        size = np.tile(np.abs(x[..., :32]) + np.abs(x[..., 32:]), 2)
    err = np.abs(got.float().numpy() - ref)
    bound = 2.0 ** -8 * np.abs(ref) + 3e-6 * (1 + 2.0 ** -8) * size
    assert (err <= bound).all(), float((err - bound).max())


def _inputs(tokens, heads, seed, axes=1, far=0):
    """q_pe and k_pe as slices of wider projections, positions [axes, T]."""
    q = _bf16((tokens, heads, 192), seed)
    kv = _bf16((tokens, 576), seed + 1)
    rng = np.random.default_rng(seed)
    pos = rng.integers(0, 5000, (axes, tokens)) + far
    return q, kv, torch.from_numpy(pos.astype(np.int32))


SECTIONS = {1: [32], 2: [12, 20], 3: [8, 12, 12]}


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens,heads,page,axes,far", [
    (1, 1, 1, 1, 0), (1, 128, 64, 3, 0), (5, 7, 7, 2, 100000), (33, 16, 16, 1, 2 ** 31 - 6000), (130, 17, 64, 3, 10 ** 6),
    (70, 33, 128, 2, 0), (3000, 1, 16, 1, 0), (257, 128, 64, 1, -5000)])
def test_append(lib, tokens, heads, page, axes, far, fp8, interleaved):
    require_gpu()
    q, kv, pos = _inputs(tokens, heads, 7 * tokens + heads, axes, far)
    pages = -(-tokens // page) + 2
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(tokens))[:tokens].to(torch.int32)
    if tokens > 4:
        slots[1], slots[2], slots[3] = -1, pages * page, 2 ** 31 - 1  # not written
    qd, kvd = q.cuda(), kv.cuda()
    args = (qd[..., 128:], kvd[:, :512], kvd[:, 512:], pos.cuda(), torch.from_numpy(FREQ).cuda(), slots.cuda())
    kw = dict(sections=SECTIONS[axes], interleaved=interleaved)
    if fp8:
        before = torch.randint(0, 256, (pages, page, 656), generator=torch.Generator().manual_seed(1),
                               dtype=torch.uint8)
        cache = before.cuda()
        q_out = lib.mla_rope_append_fp8(*args, cache, **kw)
        got = cache.cpu().view(-1, 656)
        lat, rope = got[:, :528], got[:, 528:].contiguous().view(torch.bfloat16)
        want = before.view(-1, 656)[:, :528].clone()
        rope0 = before.view(-1, 656)[:, 528:].contiguous().view(torch.bfloat16)
    else:
        ckv0, rope0 = _bf16((pages, page, 512), 3), _bf16((pages, page, 64), 4)
        ckv, kpe = ckv0.cuda(), rope0.cuda()
        q_out = lib.mla_rope_append(*args, ckv, kpe, **kw)
        lat, rope = ckv.cpu().view(-1, 512), kpe.cpu().view(-1, 64)
        want, rope0 = ckv0.view(-1, 512).clone(), rope0.view(-1, 64)
    _rope_close(q_out.cpu(), q[..., 128:], pos.numpy(), SECTIONS[axes], interleaved)
    kept = torch.nonzero((slots >= 0) & (slots < pages * page))[:, 0]
    at = slots[kept].long()
    if fp8:
        codes, scales = co.quantise(kv[kept, :512].float().numpy())
        want[at] = torch.cat([torch.from_numpy(codes), torch.from_numpy(scales).view(torch.uint8)], 1)
    else:
        want[at] = kv[kept, :512]
    assert torch.equal(lat.view(torch.uint8), want.view(torch.uint8))  # written tokens, and every other byte as it was
    _rope_close(rope[at][:, None], kv[kept][:, None, 512:], pos.numpy()[:, kept.numpy()], SECTIONS[axes], interleaved)
    others = torch.ones(pages * page, dtype=torch.bool)
    others[at] = False
    assert torch.equal(rope[others].view(torch.int16), rope0[others].view(torch.int16))


def test_append_in_place_without_queries_and_expanded_inputs(lib):
    require_gpu()
    q, kv, pos = _inputs(9, 5, 11)
    f, slots = torch.from_numpy(FREQ).cuda(), torch.arange(9, dtype=torch.int32).cuda()
    ckv, kpe = torch.zeros(9, 1, 512, dtype=torch.bfloat16).cuda(), torch.zeros(9, 1, 64, dtype=torch.bfloat16).cuda()
    kvd = kv.cuda()
    own = q[..., :64].contiguous().cuda()
    out = lib.mla_rope_append(own, kvd[:, :512], kvd[:, 512:], pos[0].cuda(), f, slots, ckv, kpe, q_out=own)
    assert out.data_ptr() == own.data_ptr()
    _rope_close(own.cpu(), q[..., :64], pos.numpy(), [32], True)
    assert lib.mla_rope_append(None, kvd[:, :512], kvd[:, 512:], pos.cuda(), f, slots, ckv, kpe) is None
    one = _bf16((1, 5, 64), 5).cuda().expand(9, 5, 64)  # one query for every position
    out = lib.mla_rope_append(one, kvd[:, :512], kvd[:, 512:], pos.cuda(), f, slots, ckv, kpe)
    _rope_close(out.cpu(), one.cpu(), pos.numpy(), [32], True)
    assert torch.equal(ckv.view(9, 512).cpu(), kv[:, :512])


def test_append_fp8_extreme_values(lib):
    """Zero tiles, values that are not finite, the largest and smallest bf16 numbers."""
    require_gpu()
    kv = _bf16((6, 576), 21)
    kv[0, :128] = 0
    kv[1, 3], kv[1, 4], kv[1, 200] = float("inf"), float("-inf"), float("nan")
    kv[2, :512] = torch.finfo(torch.bfloat16).max
    kv[3, :512] = 9.2e-41  # the smallest subnormal number
    kv[4, 5], kv[4, 6] = torch.finfo(torch.bfloat16).max, 1e-30
    kv[5, 128:256] = float("nan")
    cache = torch.zeros(1, 8, 656, dtype=torch.uint8).cuda()
    d = kv.cuda()
    lib.mla_rope_append_fp8(None, d[:, :512], d[:, 512:], torch.zeros(6, dtype=torch.int32).cuda(),
                            torch.from_numpy(FREQ).cuda(), torch.arange(6, dtype=torch.int32).cuda(), cache)
    got = cache.cpu()[0, :6]
    codes, scales = co.quantise(kv[:, :512].float().numpy())
    want = torch.from_numpy(codes)
    nan = (want & 0x7F) == 0x7F
    assert torch.equal((got[:, :512] & 0x7F) == 0x7F, nan)
    assert torch.equal(got[:, :512][~nan], want[~nan])
    assert torch.equal(got[:, 512:528].contiguous().view(torch.float32), torch.from_numpy(scales))
    assert torch.equal(got[:, 528:].contiguous().view(torch.bfloat16), kv[:, 512:])  # position 0: unchanged


def test_append_fp8_every_magnitude(lib):
    """Tiles of every bf16 exponent, values spread over 30 binades below their largest, zeros of
    both signs: the bytes are those of the IEEE quotient."""
    require_gpu()
    g = torch.Generator().manual_seed(51)
    kv = torch.randn(254 * 4, 576, generator=g)
    spread = torch.randint(-30, 1, kv.shape, generator=g)
    exponent = torch.arange(-126, 128).repeat_interleave(4)[:, None]
    kv = torch.ldexp(kv.clamp(-1.9, 1.9), (spread + exponent).clamp(min=-140)).to(torch.bfloat16)
    kv[:, 7], kv[:, 8] = 0.0, -0.0
    assert torch.isfinite(kv).all()
    n = kv.shape[0]
    cache = torch.zeros(1, n, 656, dtype=torch.uint8).cuda()
    d = kv.cuda()
    lib.mla_rope_append_fp8(None, d[:, :512], d[:, 512:], torch.zeros(n, dtype=torch.int32).cuda(),
                            torch.from_numpy(FREQ).cuda(), torch.arange(n, dtype=torch.int32).cuda(), cache)
    codes, scales = co.quantise(kv[:, :512].float().numpy())
    got = cache.cpu()[0]
    assert torch.equal(got[:, 512:528].contiguous().view(torch.float32), torch.from_numpy(scales))
    assert torch.equal(got[:, :512], torch.from_numpy(codes))


@pytest.mark.parametrize("n", [0, 1, 3, 4, 5, 129, 5000])
@pytest.mark.parametrize("fp8", [False, True])
def test_gather(lib, n, fp8):
    require_gpu()
    pages, page = 40, 7
    g = torch.Generator().manual_seed(n)
    slots = torch.randint(0, pages * page, (n,), generator=g, dtype=torch.int32)
    if n > 3:
        slots[0], slots[2], slots[3] = -1, pages * page, slots[1]
    ok = (slots >= 0) & (slots < pages * page)
    at = slots.clamp(0, pages * page - 1).long()
    if fp8:
        codes = torch.randint(0, 256, (pages * page, 512), generator=g).to(torch.uint8)
        scale = torch.rand(pages * page, 4, generator=g) * 3 - 1
        kpe = _bf16((pages * page, 64), 2)
        kv = torch.cat([codes, scale.view(torch.uint8), kpe.view(torch.uint8)], 1).view(pages, page, 656).contiguous()
        deq, _ = oracle.dequantize_fp8_cache(kv.numpy())
        ref = torch.from_numpy(np.asarray(deq)).reshape(-1, 512).to(torch.bfloat16)[at]
        call = lambda **kw: lib.mla_cache_gather_fp8(kv.cuda(), slots.cuda(), **kw)  # noqa: E731
    else:
        ckv, kpe = _bf16((pages, page, 512), 3), _bf16((pages, page, 64), 4)
        ref = ckv.view(-1, 512)[at]
        call = lambda **kw: lib.mla_cache_gather(ckv.cuda(), kpe.cuda(), slots.cuda(), **kw)  # noqa: E731
    ref_pe = kpe.view(-1, 64)[at].clone()
    ref[~ok], ref_pe[~ok] = 0, 0
    out, out_pe = call()
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(ref))
    fine = ~torch.isnan(ref)
    assert torch.equal(out.cpu()[fine], ref[fine]) and torch.equal(out_pe.cpu(), ref_pe)
    # Rows at or past the count stay as they were.
    keep = torch.full((n, 512), 7.0, dtype=torch.bfloat16).cuda()
    keep_pe = torch.full((n, 64), 7.0, dtype=torch.bfloat16).cuda()
    k = n // 2
    call(ckv_out=keep, kpe_out=keep_pe, count=torch.tensor([k], dtype=torch.int32).cuda())
    assert (keep[k:] == 7).all() and (keep_pe[k:] == 7).all()
    assert torch.equal(keep_pe[:k].cpu(), ref_pe[:k])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [1, 3, 16, 64, 100])
def test_copy_pages(lib, page, fp8):
    require_gpu()
    pages = 50
    src = torch.tensor([3, 40, -1, 7, 9, 11, 50, 12, 13], dtype=torch.int32)
    dst = torch.tensor([4, 0, 5, -1, 9, 12 + 30, 6, 50, 20], dtype=torch.int32)
    tokens = torch.tensor([page, 1, page, page, page, max(1, page // 2), page, page, 2 * page], dtype=torch.int32)
    caches = [torch.randint(0, 256, (pages, page, b), dtype=torch.uint8, generator=torch.Generator().manual_seed(b))
              for b in ((656,) if fp8 else (1024, 128))]
    for use_tokens in (False, True):
        for count in (None, 2):
            dev = [c.cuda() for c in caches]
            kw = dict(tokens=tokens.cuda() if use_tokens else None,
                      count=None if count is None else torch.tensor([count], dtype=torch.int32).cuda())
            if fp8:
                lib.mla_cache_copy_pages_fp8(*dev, src.cuda(), dst.cuda(), **kw)
            else:
                lib.mla_cache_copy_pages(*[d.view(torch.bfloat16) for d in dev], src.cuda(), dst.cuda(), **kw)
            for c, d in zip(caches, dev):
                want = c.clone()
                for i in range(9 if count is None else count):
                    s, t = int(src[i]), int(dst[i])
                    if 0 <= s < pages and 0 <= t < pages:
                        n = min(int(tokens[i]), page) if use_tokens else page
                        want[t, :n] = c[s, :n]
                assert torch.equal(d.cpu(), want)


def test_slots_past_two_gigabytes(lib):
    """Byte offsets beyond 32 bits: the last slots of a cache of 4.6 million tokens."""
    require_gpu()
    pages, page = 71500, 64  # 4.7 GB of latents
    ckv = torch.empty(pages, page, 512, dtype=torch.bfloat16, device="cuda")
    kpe = torch.empty(pages, page, 64, dtype=torch.bfloat16, device="cuda")
    kv = _bf16((4, 576), 31).cuda()
    last = pages * page - 1
    slots = torch.tensor([last, last - 64, 5, 2 ** 22], dtype=torch.int32).cuda()
    lib.mla_rope_append(None, kv[:, :512], kv[:, 512:], torch.zeros(4, dtype=torch.int32).cuda(),
                        torch.from_numpy(FREQ).cuda(), slots, ckv, kpe)
    lib.mla_cache_copy_pages(ckv, kpe, torch.tensor([pages - 1], dtype=torch.int32).cuda(),
                             torch.tensor([pages - 3], dtype=torch.int32).cuda())
    slots[0] -= 128
    a, b = lib.mla_cache_gather(ckv, kpe, slots)
    assert torch.equal(a, kv[:, :512]) and torch.equal(b, kv[:, 512:])


def test_python_refusals(lib):
    require_gpu()
    q, kv, pos = _inputs(4, 2, 41)
    q, kv, pos, f = q.cuda(), kv.cuda(), pos.cuda(), torch.from_numpy(FREQ).cuda()
    slots = torch.arange(4, dtype=torch.int32).cuda()
    ckv, kpe = torch.zeros(2, 4, 512, dtype=torch.bfloat16).cuda(), torch.zeros(2, 4, 64, dtype=torch.bfloat16).cuda()

    def call(q_pe=q[..., 128:], lat=kv[:, :512], rope=kv[:, 512:], p=pos, freq=f, s=slots, c=ckv, **kw):
        return lib.mla_rope_append(q_pe, lat, rope, p, freq, s, c, kpe, **kw)

    for kw in (dict(lat=kv[:, :500]), dict(rope=kv[:3, 512:]), dict(p=pos[:, :3]), dict(p=pos.expand(2, 4).contiguous()),
               dict(freq=f[:31].contiguous()), dict(s=slots[:3].contiguous()), dict(sections=[16, 16]),
               dict(q_pe=q[..., ::3]), dict(q_out=torch.empty(4, 2, 64, dtype=torch.bfloat16)),
               dict(q_pe=q[:3, :, 128:]), dict(c=ckv[:, :, :256])):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(p=pos.long()), dict(lat=kv[:, :512].half()), dict(freq=f.double()), dict(s=slots.long())):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(lib.MlaError):
        call(sections=[31])
    with pytest.raises(lib.MlaError):
        call(lat=_bf16((4, 520), 1).cuda()[:, 4:516])  # rows that start off the 16-byte grid
