"""GPU parity of the decoding operators with their fp64 oracle.

Tolerances (u = 2^-24, one fp32 rounding; a bf16 rounding is off by at most 2^-8 of the
value, an e4m3 one by 2^-4 or, below its smallest normal, by 2^-10):
- rotation: sine and cosine are off by at most 2^-21 (reduced angle in fp32: pi * 2^-24,
  the function itself a few u); two products and a sum add 3 u of |x1| + |x2|.
- logits: C products summed in fp32, each step off by at most 2u of the running sum of
  magnitudes (the tensor core may cut instead of round): |dx| <= 2 C u scale sum|q k|,
  plus 8 u |x| for the scalings; e4m3 adds 2^-25 of the largest q element per product.
- weights p = exp(x - m) / l: relative error 2 |dx| + 2^-20 (hardware exponential).
- o: sum p |v| times (that + 2^-16 for the split weights), then one bf16 rounding.
- lse: |dx| + 2^-20 + 4 u |lse|.  acc: sum of p's errors + 2u |acc| + u.
"""
import math

import numpy as np
import pytest
import torch

from oracle import decode_oracle as do
from tests.gpu_util import poisoned

pytestmark = pytest.mark.gpu

xa = pytest.importorskip("block_sparse_long_04_b200")

U = 2.0 ** -24
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield
    assert xa.xattn_get_device_error() == xa.XATTN_OK


def f64(t):
    return t.detach().double().cpu().numpy()


def raw(t):
    """A tensor's bits, for exact comparisons (NaN included)."""
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


# ------------------------------------------------------------------- rope
def _rope_case(seed, B, Hq, Hkv, M, C, sections, far=0):
    g = torch.Generator().manual_seed(seed)
    pairs = sum(sections)
    x = torch.randn(B, Hq + Hkv, M, C, generator=g).bfloat16().cuda()
    pos = torch.randint(0, 64, (B, M, len(sections)), generator=g).int() + far
    f = torch.cat([10000.0 ** (-torch.arange(n, dtype=torch.float64) / max(n, 1)) for n in sections])
    return x[:, :Hq], x[:, Hq:], pos.cuda(), f.cuda(), pairs


def _check_rope(got, x, pos, f, sections, interleaved, inverse):
    x = f64(x)
    pos = np.broadcast_to(pos.cpu().numpy(), (x.shape[0],) + tuple(pos.shape[-2:]))
    want = do.rope(x, pos, f64(f), sections, interleaved, inverse)
    P = sum(sections)
    mag = np.zeros_like(x)
    i = np.arange(P)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + P)
    mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    tol = 2.0 ** -8 * np.abs(want) + mag * (2.0 ** -21 + 3 * U) * (1 + 2.0 ** -8)
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), f"{(err - tol).max()}"
    np.testing.assert_array_equal(f64(got)[..., 2 * P:], x[..., 2 * P:])     # passed through


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,M,C,sections,far", [
    (1, 1, 1, 1, 64, (32,), 0),
    (2, 4, 2, 33, 128, (64,), 0),
    (3, 7, 7, 5, 64, (8,), 0),             # an eighth of the pairs
    (1, 32, 8, 17, 128, (16, 24, 24), 0),  # time, height, width
    (2, 3, 1, 40, 128, (5, 0, 11, 8), 0),  # four axes, one of them empty, odd borders
    (1, 4, 1, 300, 64, (20, 4), 1000),
    (1, 2, 2, 19, 128, (64,), 2 ** 30),    # far positions need the 64-bit angle
    (2, 2, 1, 2500, 64, (32,), 262144),    # 16-token tiles, the last one ragged
])
def test_rope(B, Hq, Hkv, M, C, sections, far, interleaved, inverse):
    q, k, pos, f, _ = _rope_case(B * 100 + M, B, Hq, Hkv, M, C, sections, far)
    rot = xa.Rotary(f, sections, interleaved)
    qo, ko = poisoned((B, Hq, M, C), torch.bfloat16), poisoned((B, Hkv, M, C), torch.bfloat16)
    xa.xattn_rope(q, k, pos, rot, qo, ko, inverse=inverse)
    _check_rope(qo, q, pos, f, sections, interleaved, inverse)
    _check_rope(ko, k, pos, f, sections, interleaved, inverse)


def test_rope_negative_positions_shared_positions_and_no_keys():
    q, _, pos, f, _ = _rope_case(5, 2, 3, 1, 9, 128, (24, 40))
    pos = (pos[0] - 5000).contiguous()
    rot = xa.Rotary(f, (24, 40))
    qo = poisoned(q.shape, torch.bfloat16)
    xa.xattn_rope(q, None, pos, rot, qo, None)
    _check_rope(qo, q, pos[None], f, (24, 40), False, False)


def test_rope_strided_in_place_and_back():
    """A slice of a fused projection, outputs in another layout, in place, and the inverse."""
    B, M, Hq, Hkv, C = 2, 37, 6, 2, 128
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(B, M, Hq + 2 * Hkv, C, generator=g).bfloat16().cuda()
    q, k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
    pos = torch.arange(M, dtype=torch.int32, device="cuda")[:, None].contiguous()
    rot = xa.Rotary.make((64,))
    dense_q, dense_k = poisoned(q.shape, torch.bfloat16), poisoned(k.shape, torch.bfloat16)
    xa.xattn_rope(q.contiguous(), k.contiguous(), pos, rot, dense_q, dense_k)
    out = poisoned((B, M, Hq + Hkv, C), torch.bfloat16)
    xa.xattn_rope(q, k, pos, rot, out[:, :, :Hq].transpose(1, 2), out[:, :, Hq:].transpose(1, 2))
    assert torch.equal(out[:, :, :Hq].transpose(1, 2), dense_q)
    assert torch.equal(out[:, :, Hq:].transpose(1, 2), dense_k)
    before = qkv.clone()
    xa.xattn_rope(q, k, pos, rot, q, k)
    assert torch.equal(q, dense_q) and torch.equal(k, dense_k)
    assert torch.equal(qkv[:, :, Hq + Hkv:], before[:, :, Hq + Hkv:])
    xa.xattn_rope(q, k, pos, rot, q, k, inverse=True)
    # two bf16 roundings apart from the start: 2^-8 of a pair's length each
    far = (f64(qkv) - f64(before))
    size = np.hypot(f64(before)[..., :64], f64(before)[..., 64:])
    assert (np.abs(far) <= np.concatenate([size, size], -1) * 2.0 ** -8 * 2.1).all()


def test_rope_gradient_against_differences():
    """d/dx <g, rope(x)> by the inverse call against central differences of the forward call;
    the step is a power of two, so that only the outputs' bf16 roundings count."""
    B, H, M, C, sections = 1, 1, 3, 64, (8, 8)
    x, _, pos, f, _ = _rope_case(11, B, H, 1, M, C, sections)
    rot = xa.Rotary(f, sections)
    g = torch.zeros_like(x)
    g[0, 0, 1] = 1.0
    grad = poisoned(g.shape, torch.bfloat16)
    xa.xattn_rope(g.contiguous(), None, pos, rot, grad, None, inverse=True)
    for i in (0, 5, 17, 31, 32, 63):
        y = []
        for step in (64.0, -64.0):
            z = torch.zeros_like(x)
            z[0, 0, 1, i] = step
            o = poisoned(z.shape, torch.bfloat16)
            xa.xattn_rope(z, None, pos, rot, o, None)
            y.append(f64(o))
        num = ((y[0] - y[1]) * f64(g)).sum() / 128.0
        # each of the (up to two) outputs is off by 2^-8 of at most 1, the gradient by 2^-8
        assert abs(num - f64(grad)[0, 0, 1, i]) <= 2 * 2.0 ** -8 + 2.0 ** -8 * 1.5


# ------------------------------------------------------------------ caches
def make_cache(seed, lens, Hkv, C, page, e4m3=False, eviction=True, spare=3, table_fill=-1, slack=0):
    """A cache with its pages in random order. Rows that no sequence uses hold NaN (in pages,
    behind a sequence's end, and in free pages), and free table entries hold table_fill."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    P = sum(need) + spare
    order = torch.randperm(P, generator=g)[:sum(need)].int()
    width = max(1, max(need)) + slack
    table = torch.full((len(lens), width), table_fill, dtype=torch.int32)
    at = 0
    k = torch.full((P, Hkv, page, C), float("nan"))
    v, acc = k.clone(), torch.full((P, Hkv, page), float("nan"))
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
        for i in range(n):
            m = min(page, lens[b] - i * page)
            k[table[b, i], :, :m] = torch.randn(Hkv, m, C, generator=g)
            v[table[b, i], :, :m] = torch.randn(Hkv, m, C, generator=g)
            acc[table[b, i], :, :m] = torch.rand(Hkv, m, generator=g)
    scales = (None, None)
    if e4m3:
        scales = (torch.rand(Hkv, generator=g) * 0.02 + 0.01, torch.rand(Hkv, generator=g) * 0.02 + 0.01)
        k = (k / scales[0][:, None, None]).clamp(-448, 448).to(E4M3)
        v = (v / scales[1][:, None, None]).clamp(-448, 448).to(E4M3)
        scales = (scales[0].cuda(), scales[1].cuda())
    else:
        k, v = k.bfloat16(), v.bfloat16()
    return xa.PagedCache(k.cuda(), v.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                         *scales, acc=acc.cuda() if eviction else None,
                         ordinal=torch.zeros(P, Hkv, page, dtype=torch.int32).cuda() if eviction else None)


def to_oracle(c):
    z = np.zeros(c.k_pages.shape[:3])
    return dict(k=f64(c.k_pages), v=f64(c.v_pages), acc=f64(c.acc) if c.acc is not None else z,
                ordinal=c.ordinal.cpu().numpy().astype(np.int64) if c.ordinal is not None else z.astype(int),
                table=c.page_table.cpu().numpy(), lens=c.lens.cpu().numpy(),
                k_scale=None if c.k_scale is None else f64(c.k_scale),
                v_scale=None if c.v_scale is None else f64(c.v_scale))


def clone_cache(c):
    def cp(t):
        return None if t is None else t.clone()
    return xa.PagedCache(*[cp(t) for t in (c.k_pages, c.v_pages, c.page_table, c.lens, c.k_scale,
                                           c.v_scale, c.acc, c.ordinal)])


def same_cache(a, b):
    return all(torch.equal(raw(x), raw(y)) for x, y in (
        (a.k_pages, b.k_pages), (a.v_pages, b.v_pages)) + (
        () if a.acc is None else ((a.acc, b.acc), (a.ordinal, b.ordinal))))


# ------------------------------------------------------------------ append
APPENDS = [
    # lens (after the append), n_new, T, Hq, Hkv, C, page
    ([1], [1], 1, 4, 1, 128, 16),
    ([130, 1, 16], [1, 1, 1], 1, 8, 2, 128, 16),
    ([5, 64, 200, 33], [5, 0, 77, 1], 77, 6, 3, 64, 32),      # a padded batch, one without a new token
    ([700], None, 300, 4, 4, 128, 128),
    ([6000, 4100], [4099, 4100], 4100, 2, 1, 64, 64),         # 16-token tiles
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("lens,new,T,Hq,Hkv,C,page", APPENDS)
def test_append(lens, new, T, Hq, Hkv, C, page, rope, e4m3):
    B = len(lens)
    c = make_cache(7 + T, lens, Hkv, C, page, e4m3)
    before, want = clone_cache(c), to_oracle(c)
    g = torch.Generator().manual_seed(T)
    qkv = torch.randn(B, T, Hq + 2 * Hkv, C, generator=g).bfloat16().cuda()
    q, k, v = (x.transpose(1, 2) for x in qkv.split([Hq, Hkv, Hkv], 2))
    n_new = torch.tensor([T] * B if new is None else new, dtype=torch.int32).cuda()
    seen = c.lens + 1000
    args = dict(n_new=None if new is None else n_new, seen=seen)
    kk = f64(k)
    if rope:
        pos = ((seen - n_new)[:, None] + torch.arange(T, device="cuda")).int()[..., None].contiguous()
        rot = xa.Rotary.make((C // 2,))
        qo = poisoned(q.shape, torch.bfloat16)
        xa.xattn_rope_append(q, k, v, pos, rot, c, qo, **args)
        kk = do.rope(kk, pos.cpu().numpy(), f64(rot.inv_freq), (C // 2,))
        alone = poisoned(q.shape, torch.bfloat16)
        xa.xattn_rope(q, None, pos, rot, alone, None)
        for b in range(B):
            n = int(n_new[b])
            assert torch.equal(qo[b, :, :n], alone[b, :, :n])
            assert torch.isnan(qo[b, :, n:]).all()                 # padding: left as it was
    else:
        xa.xattn_cache_append(k, v, c, **args)
    nn = n_new.cpu().numpy()
    want = do.cache_append(want, kk, f64(v), nn, seen.cpu().numpy())
    touched = np.zeros(c.k_pages.shape[:3], bool)
    for b in range(B):
        for s in range(lens[b] - int(nn[b]), lens[b]):
            pg, r = do.cache_slot(want, b, s)
            touched[pg, :, r] = True
    for name, got in (("k", c.k_pages), ("v", c.v_pages)):
        w, y = want[name][touched], f64(got)[touched]
        if name == "k" and rope:
            # a rotated element is off by (2^-21 + 3u)(|x1| + |x2|) before it is stored
            near = 16.0 * (2.0 ** -21 + 3 * U) / (1.0 if not e4m3 else float(c.k_scale.min()))
        else:
            near = 0.0
        if e4m3:
            tol = np.maximum(2.0 ** -4 * np.abs(w), 2.0 ** -10) * (1 + 2 * U) + near + U * np.abs(w)
        else:
            tol = 2.0 ** -8 * np.abs(w) + near if near else 0.0 * w
        assert (np.abs(y - w) <= tol).all()
    t = torch.from_numpy(touched).cuda()
    assert (c.acc[t] == 0).all()
    np.testing.assert_array_equal(c.ordinal.cpu().numpy()[touched], want["ordinal"][touched])
    # nothing else was written
    for a, b2 in ((c.k_pages, before.k_pages), (c.v_pages, before.v_pages), (c.acc, before.acc),
                  (c.ordinal, before.ordinal)):
        assert torch.equal(raw(a)[~t], raw(b2)[~t])


def test_append_e4m3_special_values():
    """Saturation, infinities, NaN, signed zero and halves of the smallest step, against
    torch's conversion of the same quotients."""
    vals = torch.tensor([0.0, -0.0, 448, 449, 464, 480, 1e30, float("inf"), -float("inf"), float("nan"),
                         2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -11, -2.0 ** -11, 1.0625, 1.1875] * 4)
    c = xa.PagedCache.allocate(1, 2, 64, 1, 1, page=16, dtype=E4M3, k_scale=torch.tensor([1.0, 3.0]).cuda(),
                               v_scale=torch.tensor([0.37, 1e-3]).cuda())
    c.lens.fill_(1)
    x = vals.bfloat16().cuda().view(1, 1, 1, 64).expand(1, 2, 1, 64)       # shared rows: stride 0
    xa.xattn_cache_append(x, x, c)
    for pages, sc in ((c.k_pages, c.k_scale), (c.v_pages, c.v_scale)):
        want = (x[0, :, 0].float() / sc[:, None]).clamp(-448, 448).to(E4M3)
        nan = torch.isnan(want.float())
        assert torch.equal(torch.isnan(pages[0, :, 0].float()), nan)
        assert torch.equal(raw(pages[0, :, 0])[~nan], raw(want)[~nan])


def test_append_e4m3_quotients_of_every_value():
    """Every finite bf16 value over scales of many sizes, those among them whose quotients lie
    next to the middle of two e4m3 values, bit for bit against torch's division and conversion."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[torch.isfinite(x.float())].view(-1, 64)
    mids = [1 + (2 * i + 1) / 16 for i in range(8)]
    f32 = torch.float32
    scales = torch.cat([torch.rand(16, generator=torch.Generator().manual_seed(0)) * 0.05 + 1e-3,
                        torch.tensor([1.0, 0.5, 3.0, 1 / 3, 448.0, 1 / 448, 2.0 ** -126, 2.0 ** -130, 2.0 ** 127,
                                      3.0e38, 1e-30, 1e30], dtype=f32),
                        torch.tensor([a / m for m in mids for a in (1.0, 1.0078125, 1.9921875)], dtype=f32)])
    for s in torch.stack([scales, scales.flip(0)], 1):
        c = xa.PagedCache.allocate(1, 2, 64, x.shape[0] // 64 + 1, x.shape[0] // 64 + 1, page=64, dtype=E4M3,
                                   k_scale=s.cuda(), v_scale=s.flip(0).contiguous().cuda())
        c.lens.fill_(x.shape[0])
        rows = x.cuda()[None, None].expand(1, 2, -1, -1)
        xa.xattn_cache_append(rows, rows, c)
        for pages, sc in ((c.k_pages, s), (c.v_pages, s.flip(0))):
            for h in range(2):
                want = (x.float() / sc[h]).clamp(-448, 448).to(E4M3)
                got = pages[:, h].reshape(-1, 64)[:x.shape[0]].cpu()
                assert torch.equal(raw(got), raw(want)), sc[h]


# ------------------------------------------------------------------ decode
def run_decode(c, q, scale, weights=False, acc_out=None, stream=None):
    B, Hq, C = q.shape
    o, lse = poisoned((B, Hq, C), torch.bfloat16), poisoned((B, Hq))
    ws = poisoned(xa.xattn_decode_workspace_size(c, Hq, weights), torch.uint8)
    xa.xattn_decode_attn(q, c, scale, o, ws, lse=lse, weights=weights, acc_out=acc_out, stream=stream)
    return o, lse


def check_decode(c, q, scale, o, lse, acc_before=None, acc_after=None):
    oc, qd = to_oracle(c), f64(q)
    wo, wl, ww = do.decode_attention(qd, oc, scale)
    B, Hq, C = qd.shape
    Hkv = c.Hkv
    o, lse = f64(o), f64(lse)
    for b in range(B):
        n = int(oc["lens"][b])
        if n == 0:
            assert (o[b] == 0).all() and np.isneginf(lse[b]).all()
            continue
        for h in range(Hkv):
            k, v = do.cache_rows(oc, "k", b, h), do.cache_rows(oc, "v", b, h)
            acc_tol = 0
            for hq in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                x = scale * (k @ qd[b, hq])
                dx = (2 * C * U + (2.0 ** -24 if c.k_scale is not None else 0)) * scale * (
                    np.abs(k) @ np.abs(qd[b, hq])) + 8 * U * np.abs(x)
                if c.k_scale is not None:
                    dx = dx + 2.0 ** -25 * scale * np.abs(qd[b, hq]).max() * np.abs(k).sum(1)
                dx = dx.max()
                p = np.exp(x - wl[b, hq])
                rel = 2 * dx + 2.0 ** -20
                tol = 2.0 ** -8 * np.abs(wo[b, hq]) + (p @ np.abs(v)) * (rel + 2.0 ** -16) * 1.01
                assert (np.abs(o[b, hq] - wo[b, hq]) <= tol).all(), (b, hq)
                assert abs(lse[b, hq] - wl[b, hq]) <= dx + 2.0 ** -20 + 4 * U * abs(wl[b, hq])
                acc_tol = acc_tol + p * rel
            if acc_after is not None:
                where = [do.cache_slot(oc, b, s) for s in range(n)]
                old = np.array([acc_before[pg, h, r] for pg, r in where])
                new = np.array([acc_after[pg, h, r] for pg, r in where])
                assert (np.abs(new - (old + ww[b][h])) <= acc_tol + 2 * U * np.abs(new) + U).all()


DECODES = [
    # lens, Hq, Hkv, C, page
    ([1], 1, 1, 64, 16),
    ([1, 2, 15, 16, 17, 63, 64, 65], 4, 2, 128, 16),
    ([0], 4, 1, 128, 64),
    ([0, 0, 5, 0], 2, 2, 64, 32),
    ([777], 32, 8, 128, 16),
    ([1000, 3, 0, 250], 12, 4, 128, 64),
    ([129, 400], 7, 7, 64, 128),
    ([333], 16, 1, 128, 32),          # 16 heads per kv head
    ([200, 90], 9, 1, 64, 16),        # 9: the second head tile holds one
    ([150], 34, 2, 128, 128),         # 17: two tiles of 16
    ([100, 31], 40, 1, 64, 64),       # 40: three tiles, the last of eight
    ([2100], 128, 1, 64, 16),
    ([5] * 37, 3, 3, 64, 16),         # more sequences than a warp
    ([20000], 1, 1, 64, 128),         # more tiles than CTAs
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,C,page", DECODES)
def test_decode(lens, Hq, Hkv, C, page, weights, e4m3):
    c = make_cache(len(lens) + sum(lens), lens, Hkv, C, page, e4m3, slack=2)
    g = torch.Generator().manual_seed(Hq)
    q = (2 * torch.randn(len(lens), Hq, C, generator=g)).bfloat16().cuda()
    scale = 1 / math.sqrt(C)
    before = clone_cache(c)
    if weights:
        acc_out = c.acc.clone()
        o, lse = run_decode(c, q, scale, True, acc_out)
        check_decode(c, q, scale, o, lse, f64(before.acc), f64(acc_out))
        used = np.zeros(c.acc.shape, bool)
        for b, n in enumerate(lens):
            for s in range(n):
                pg, r = do.cache_slot(dict(table=c.page_table.cpu().numpy(), k=c.k_pages), b, s)
                used[pg, :, r] = True
        free = ~torch.from_numpy(used).cuda()
        assert torch.equal(raw(acc_out)[free], raw(before.acc)[free])     # slots not in use
        assert same_cache(c, before)
        o2, lse2 = run_decode(c, q, scale, True)                          # in place: the same
        assert torch.equal(raw(c.acc), raw(acc_out))
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
    else:
        o, lse = run_decode(c, q, scale)
        check_decode(c, q, scale, o, lse)
        assert same_cache(c, before)
    # every run gives the same bits
    o2, lse2 = run_decode(c, q, scale)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("Hq,Hkv,C,first", [(4, 1, 128, 5), (4, 2, 64, 1333), (16, 1, 128, 5)])
@pytest.mark.parametrize("octaves", [20, 30, 60, 100])
def test_decode_beside_a_slot_that_takes_nearly_all_the_weight(octaves, Hq, Hkv, C, first, e4m3):
    """One slot whose value is 0 (an attention sink) outweighs each of the others by 2^octaves,
    so the output is made of the small weights alone. The same pages serve 300 sequences, so
    that a CTA walks many tiles, and from every start. Tolerance of the output as in
    check_decode, and over e4m3 pages per slot 2^-26 of the largest weight among the 32
    neighbouring slots that are weighed together (they are held in f16, that largest one at 4
    or above, with an error of 2^-25) or 2^-112 of the head's largest; at most the weight itself."""
    n, B, scale = 2500, 300, 1 / math.sqrt(C)
    c = make_cache(21, [n], Hkv, C, 32, e4m3, eviction=False)
    g = torch.Generator().manual_seed(4)
    q = (torch.rand(1, 1, C, generator=g) + 0.5).bfloat16()     # one query: one key outweighs for every head
    k, v = c.k_pages.float(), c.v_pages.float()
    pg, r = do.cache_slot(to_oracle(c), 0, first)
    k = k * 2.0 ** -5
    k[pg, :, r] = octaves * math.log(2) / scale / q.float().sum().item()
    if e4m3:
        c.k_scale.mul_(2)            # the heavy key is below 448 scales
        k[pg, :, r] /= c.k_scale[:, None]
    v = v.abs() * 0.25 + (16.0 if e4m3 else 1.0)
    v[pg, :, r] = 0
    c.k_pages.copy_(k)
    c.v_pages.copy_(v)
    many = xa.PagedCache(c.k_pages, c.v_pages, c.page_table.expand(B, -1).contiguous(), c.lens.expand(B).contiguous(),
                         c.k_scale, c.v_scale)
    o, lse = run_decode(many, q.expand(B, Hq, C).contiguous().cuda(), scale)
    oc, qd = to_oracle(c), f64(q)[0, 0]
    wo, wl, _ = do.decode_attention(np.broadcast_to(qd, (1, Hq, C)), oc, scale)
    for hq in range(Hq):
        k, v = do.cache_rows(oc, "k", 0, hq * Hkv // Hq), do.cache_rows(oc, "v", 0, hq * Hkv // Hq)
        x = scale * (k @ qd)
        dx = (2 * C * U + (2.0 ** -24 if e4m3 else 0)) * scale * (np.abs(k) @ np.abs(qd)) + 8 * U * np.abs(x)
        if e4m3:
            dx = dx + 2.0 ** -25 * scale * np.abs(qd).max() * np.abs(k).sum(1)
        p = np.exp(x - wl[0, hq])
        assert p[first] > 0.9 and p.sum() - p[first] < 2.0 ** (14 - octaves)
        tol = 2.0 ** -8 * np.abs(wo[0, hq]) + (p @ np.abs(v)) * (2 * dx.max() + 2.0 ** -20 + 2.0 ** -16) * 1.01
        if e4m3:
            top = np.maximum.reduceat(p, np.arange(0, n, 32)).repeat(32)[:n]
            tol = tol + np.minimum(np.maximum(2.0 ** -26 * top, 2.0 ** -112 * p.max()), p) @ np.abs(v)
        assert (np.abs(f64(o)[:, hq] - wo[0, hq]) <= tol).all(), hq
        assert np.abs(wo[0, hq]).min() > 4 * tol.max()       # the outputs are not all tolerance


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("shift", [30.0, 300.0, -300.0])
def test_decode_with_far_larger_and_smaller_logits(shift, e4m3):
    """Single keys whose logits tower over (or sink below) the others, early and late in
    the sequence, so that running maxima move by more than fp32's exponent range."""
    lens, C = [700, 130], 64
    c = make_cache(5, lens, 2, C, 16, e4m3)
    g = torch.Generator().manual_seed(1)
    q = (torch.rand(2, 4, C, generator=g) + 0.5).bfloat16().cuda()
    oc = to_oracle(c)
    for b, s in ((0, 0), (0, 350), (0, 699), (1, 129)):
        pg, r = do.cache_slot(oc, b, s)
        for h in range(2):
            row = torch.full((C,), shift / (C * 0.125) * (1 + s / 7000))
            row = row / c.k_scale[h].item() if e4m3 else row
            c.k_pages[pg, h, r] = row.clamp(-448, 448).to(c.k_pages.dtype).cuda()
    o, lse = run_decode(c, q, 0.125)
    check_decode(c, q, 0.125, o, lse)


def test_decode_queries_of_every_size_e4m3():
    """The per-head power of two of the e4m3 path: zero, tiny, huge and mixed queries."""
    C = 128
    c = make_cache(9, [100], 1, C, 32, True)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(1, 6, C, generator=g)
    q[0, 0] = 0
    q[0, 1] *= 2.0 ** -120
    q[0, 2] *= 2.0 ** 60
    q[0, 3, :64] *= 2.0 ** -30
    q[0, 4, 1:] = 0
    q[0, 5] = 2.0 ** -133         # bf16 subnormals
    q = q.bfloat16().cuda()
    o, lse = run_decode(c, q, 2.0 ** -60)
    check_decode(c, q, 2.0 ** -60, o, lse)
    o, lse = run_decode(c, q[:, :2], 0.1)
    check_decode(c, q[:, :2], 0.1, o, lse)


def test_decode_infinities_and_nan_in_reach():
    """-inf logits drop out; a NaN key or value in use makes its own head NaN and no other."""
    C = 64
    c = make_cache(3, [50, 40], 2, C, 16)
    q = torch.ones(2, 4, C).bfloat16().cuda()
    t = c.page_table.cpu()
    c.k_pages[t[0, 1], 0, 3] = float("-inf")         # slot 19 of sequence 0, kv head 0
    c.v_pages[t[1, 0], 1, 5] = float("nan")          # slot 5 of sequence 1, kv head 1
    o, lse = run_decode(c, q, 0.125)
    want_cache = clone_cache(c)
    want_cache.k_pages[t[0, 1], 0, 3] = -1e30
    want_cache.v_pages[t[1, 0], 1, 5] = 0
    o2, lse2 = run_decode(want_cache, q, 0.125)
    assert torch.equal(lse, lse2)
    assert torch.isnan(o[1, 2:]).all() and not torch.isnan(o[1, :2]).any()
    assert torch.equal(o[0], o2[0]) and torch.equal(o[1, :2], o2[1, :2])
    # all logits -inf: no mass, as for an empty sequence
    c = make_cache(3, [20], 1, C, 16)
    c.k_pages.fill_(float("-inf"))
    o, lse = run_decode(c, q[:1, :2].contiguous(), 0.125, True)
    assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("lens,slot", [([1, 30], 0), ([50, 9], 19), ([20000, 5], 7777)])
@pytest.mark.parametrize("C,Hq,Hkv", [(64, 4, 2), (128, 16, 1)])
def test_decode_infinite_values_in_reach(lens, slot, C, Hq, Hkv):
    """Infinite values in use make their columns that infinity, or NaN where both signs meet;
    every other column is as if they were not there."""
    c = make_cache(31, lens, Hkv, C, 16)
    q = (0.5 * torch.randn(2, Hq, C, generator=torch.Generator().manual_seed(6))).bfloat16().cuda()
    t = c.page_table.cpu()
    inf, at = float("inf"), (int(t[0, slot // 16]), Hkv - 1, slot % 16)
    fine = clone_cache(c)
    o, lse = run_decode(fine, q, 1 / math.sqrt(C))
    want = o.clone()
    mine = slice((Hkv - 1) * Hq // Hkv, Hq)            # the query heads of that kv head
    c.v_pages[at[0], at[1], at[2], 3] = inf
    c.v_pages[at[0], at[1], at[2], C - 1] = -inf
    want[0, mine, 3], want[0, mine, C - 1] = inf, -inf
    if lens[0] > 1:                                    # infinities of both signs: NaN
        other = (slot + 5) % lens[0]
        for s, x in ((slot, inf), (other, -inf)):
            c.v_pages[int(t[0, s // 16]), Hkv - 1, s % 16, 9] = x
        want[0, mine, 9] = float("nan")
    got, lse2 = run_decode(c, q, 1 / math.sqrt(C))
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok]) and torch.equal(lse, lse2)


def test_decode_strided_queries_and_4d():
    C, lens = 128, [70, 9]
    c = make_cache(12, lens, 2, C, 16, eviction=False)
    qkv = torch.randn(2, 1, 12, C, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    q = qkv[:, :, 2:10].transpose(1, 2)              # [B, 8, 1, C]
    o = poisoned((2, 8, 1, C), torch.bfloat16)
    ws = poisoned(xa.xattn_decode_workspace_size(c, 8), torch.uint8)
    xa.xattn_decode_attn(q, c, 0.1, o, ws)
    o2, _ = run_decode(c, q[:, :, 0].contiguous(), 0.1)
    assert torch.equal(o[:, :, 0], o2)


def test_decode_shared_prefix_pages():
    """Two sequences that name the same pages (read only)."""
    C = 64
    c = make_cache(4, [64, 64], 1, C, 32, eviction=False)
    c.page_table[1] = c.page_table[0]
    q = torch.randn(1, 2, C, generator=torch.Generator().manual_seed(0)).bfloat16().cuda().expand(2, 2, C)
    o, lse = run_decode(c, q, 0.1)
    check_decode(c, q, 0.1, o, lse)
    assert torch.equal(o[0], o[1])


# ------------------------------------------------------------------- evict
def run_evict(c, budget, recent=0, sink=0, seen=None, **kw):
    ws = poisoned(max(1, xa.xattn_cache_evict_workspace_size(c, budget)), torch.uint8)
    xa.xattn_cache_evict(c, budget, ws, recent=recent, sink=sink, seen=seen, **kw)


def fill_eviction(c, seed, ties=False):
    """Random weights and ordinals in the slots in use."""
    rng = np.random.default_rng(seed)
    acc, age = f64(c.acc), c.ordinal.cpu().numpy()
    oc = to_oracle(c)
    for b, n in enumerate(oc["lens"]):
        for h in range(c.Hkv):
            w = rng.gamma(0.3, size=n).astype(np.float32)
            if ties:
                w = np.round(w * 3).astype(np.float32) / 3
            o = np.sort(rng.choice(3 * n, n, replace=False)) if n else []
            if n > 4:       # some slots out of order, as earlier evictions leave them
                i = rng.choice(n, n // 4, replace=False)
                o[np.sort(i)] = o[i]
            for s in range(n):
                pg, r = do.cache_slot(oc, b, s)
                acc[pg, h, r], age[pg, h, r] = w[s], o[s]
    c.acc.copy_(torch.from_numpy(acc.astype(np.float32)))
    c.ordinal.copy_(torch.from_numpy(age))


EVICTS = [
    # lens, Hkv, C, page, budget, recent, sink
    ([10], 1, 64, 16, 1, 0, 0),
    ([10, 3, 0, 8], 2, 128, 16, 4, 1, 1),
    ([100, 57], 2, 64, 32, 57, 20, 4),
    ([100], 1, 128, 16, 99, 0, 0),          # one slot goes
    ([100], 3, 64, 128, 100, 0, 0),         # none
    ([300, 299, 17], 2, 128, 64, 1000, 10, 0),   # a budget beyond the cache
    ([513, 512, 511], 1, 64, 16, 200, 150, 50),  # all of the budget safe
    ([2049], 1, 64, 16, 1024, 100, 4),
    ([5000, 4097], 1, 64, 128, 1500, 30, 2),     # a cluster of CTAs per row
    ([17000], 1, 64, 16, 16000, 0, 0),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("lens,Hkv,C,page,budget,recent,sink", EVICTS)
def test_evict(lens, Hkv, C, page, budget, recent, sink, ties, e4m3):
    c = make_cache(sum(lens), lens, Hkv, C, page, e4m3, slack=1)
    fill_eviction(c, budget, ties)
    seen = 3 * c.lens
    before = clone_cache(c)
    want = do.cache_evict(to_oracle(c), budget, recent, sink, seen.cpu().numpy())
    acc_out, ord_out = c.acc.clone().fill_(-3), c.ordinal.clone().fill_(-7)
    out_of_place = clone_cache(c)
    run_evict(out_of_place, budget, recent, sink, seen, acc_out=acc_out, ord_out=ord_out)
    run_evict(c, budget, recent, sink, seen)
    for name, t in (("k", c.k_pages), ("v", c.v_pages), ("acc", c.acc), ("ordinal", c.ordinal)):
        np.testing.assert_array_equal(f64(t), want[name])
    assert torch.equal(c.lens, before.lens)
    # into other arrays: the same slots 0..n-1, nothing else, and the inputs untouched
    assert torch.equal(raw(out_of_place.k_pages), raw(c.k_pages))
    assert torch.equal(raw(out_of_place.acc), raw(before.acc))
    assert torch.equal(out_of_place.ordinal, before.ordinal)
    kept = np.zeros(c.acc.shape, bool)
    for b, n in enumerate(lens):
        for s in range(min(n, budget)):
            pg, r = do.cache_slot(want, b, s)
            kept[pg, :, r] = True
    t = torch.from_numpy(kept).cuda()
    assert torch.equal(acc_out[t], c.acc[t]) and torch.equal(ord_out[t], c.ordinal[t])
    assert (acc_out[~t] == -3).all() and (ord_out[~t] == -7).all()


def test_evict_special_weights():
    """All equal, negative, signed zeros, subnormals, infinities and NaN."""
    n, C = 64, 64
    rows = [torch.zeros(n), -torch.arange(n).float(), torch.tensor([0.0, -0.0] * 32),
            torch.arange(n).float() * 2.0 ** -149,
            torch.tensor([float("inf"), 1.0, float("-inf"), float("nan")] * 16),
            torch.tensor([float("nan"), float("inf")] * 32)]
    c = make_cache(1, [n], len(rows), C, 16)
    t = c.page_table[0].cpu()
    for h, w in enumerate(rows):
        for i in range(4):
            c.acc[t[i], h] = w[i * 16:(i + 1) * 16].cuda()
            c.ordinal[t[i], h] = torch.arange(i * 16, i * 16 + 16, dtype=torch.int32).cuda()
    want = do.cache_evict(to_oracle(c), 23, 5, 3, [n])
    run_evict(c, 23, 5, 3)
    for name, x in (("k", c.k_pages), ("acc", c.acc), ("ordinal", c.ordinal)):
        np.testing.assert_array_equal(f64(x), want[name])


@pytest.mark.parametrize("n,Hkv,budget", [
    (45056, 80, 30000),      # one CTA per row, its keys in the workspace
    (131072, 2, 70001),      # a cluster per row, keys in shared memory
    (400000, 1, 399999),     # a cluster per row, keys in the workspace; one slot goes
])
def test_evict_long_rows(n, Hkv, budget):
    """Rows beyond what the oracle walks through: against a sort on the GPU."""
    page, C = 64, 64
    P = n // page
    g = torch.Generator(device="cuda").manual_seed(0)
    k = torch.empty(P, Hkv, page, C, dtype=E4M3, device="cuda")
    one = torch.ones(Hkv, device="cuda")
    acc = torch.rand(P, Hkv, page, device="cuda", generator=g)
    age = torch.arange(n, dtype=torch.int32, device="cuda").view(P, 1, page).expand(P, Hkv, page).contiguous()
    c = xa.PagedCache(k, k.clone(), torch.arange(P, dtype=torch.int32, device="cuda")[None],
                      torch.tensor([n], dtype=torch.int32, device="cuda"), one, one, acc, age)
    flat = acc.permute(1, 0, 2).reshape(Hkv, n)
    safe = torch.arange(n, device="cuda") >= n - 500
    order = torch.where(safe, float("inf"), flat).sort(dim=1, descending=True, stable=True).indices[:, :budget]
    run_evict(c, budget, 500, 0)
    got = c.ordinal.permute(1, 0, 2).reshape(Hkv, n)[:, :budget]
    assert torch.equal(got.sort(dim=1).values, order.int().sort(dim=1).values)
    w = c.acc.permute(1, 0, 2).reshape(Hkv, n)[:, :budget]
    assert torch.equal(w, flat.gather(1, got.long()))


@pytest.mark.parametrize("B,Hkv,page,max_pages,in_workspace", [
    (9, 8, 16, 2561, False),
    (9, 8, 16, 5125, True),        # clusters of 2, 4, 4, 8, 8 CTAs
    (4, 8, 32, 5121, True),
    (4, 8, 16, 10241, True),
    (1, 8, 64, 5121, True),
    (3, 1, 16, 20501, True),
])
def test_evict_with_a_table_wider_than_the_rows(B, Hkv, page, max_pages, in_workspace):
    """Tables made for long contexts, of odd lengths, over short sequences: the plan goes by the
    table, so the selection's keys lie in the workspace, in one part per CTA of a cluster. The
    same rows in a table just wide enough give the same cache."""
    lens = [200 + 37 * b for b in range(B)]
    c = make_cache(B, lens, Hkv, 64, page)
    fill_eviction(c, page)
    wide = clone_cache(c)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
    table[:, :c.max_pages] = c.page_table
    wide = xa.PagedCache(wide.k_pages, wide.v_pages, table, wide.lens, acc=wide.acc, ordinal=wide.ordinal)
    assert (xa.xattn_cache_evict_workspace_size(wide, 150) > 4 * max_pages * page * B * Hkv) == in_workspace
    want = do.cache_evict(to_oracle(c), 150, 20, 4, (3 * c.lens).cpu().numpy())
    run_evict(c, 150, 20, 4, 3 * c.lens)
    run_evict(wide, 150, 20, 4, 3 * wide.lens)
    assert same_cache(wide, c)
    for name, t in (("k", wide.k_pages), ("v", wide.v_pages), ("acc", wide.acc), ("ordinal", wide.ordinal)):
        np.testing.assert_array_equal(f64(t), want[name])


@pytest.mark.parametrize("n,Hkv,page,max_pages,budget", [
    (131000, 64, 16, 8193, 60000),     # a cluster of 2, both parts in use
    (163000, 32, 32, 5121, 100001),    # of 4
    (327700, 8, 64, 5121, 200002),     # of 8
])
def test_evict_long_rows_with_keys_in_the_workspace(n, Hkv, page, max_pages, budget):
    """Long rows in tables whose parts of the workspace are not whole multiples of 16 bytes by
    their length alone: against a sort on the GPU."""
    C, P = 64, -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.zeros(P, Hkv, page, C, dtype=E4M3, device="cuda")
    one = torch.ones(Hkv, device="cuda")
    acc = torch.rand(P, Hkv, page, device="cuda", generator=g)
    age = torch.arange(P * page, dtype=torch.int32, device="cuda").view(P, 1, page).expand(P, Hkv, page).contiguous()
    table = torch.full((1, max_pages), -1, dtype=torch.int32, device="cuda")
    table[0, :P] = torch.arange(P, dtype=torch.int32, device="cuda")
    c = xa.PagedCache(k, k.clone(), table, torch.tensor([n], dtype=torch.int32, device="cuda"), one, one, acc, age)
    flat = acc.permute(1, 0, 2).reshape(Hkv, -1)[:, :n]
    safe = torch.arange(n, device="cuda") >= n - 500
    order = torch.where(safe, float("inf"), flat).sort(dim=1, descending=True, stable=True).indices[:, :budget]
    flat = flat.clone()
    run_evict(c, budget, 500, 0)
    got = c.ordinal.permute(1, 0, 2).reshape(Hkv, -1)[:, :budget]
    assert torch.equal(got.sort(dim=1).values, order.int().sort(dim=1).values)
    w = c.acc.permute(1, 0, 2).reshape(Hkv, -1)[:, :budget]
    assert torch.equal(w, flat.gather(1, got.long()))

# ------------------------------------------------- the operators as a user runs them
def test_prefill_append_decode_evict_decode():
    """A prompt through the prefill, its keys into the cache, decoding steps that rotate,
    append, attend and accumulate, an eviction, and more steps: each step's output against
    the oracle's on the cache as it then is, and the first one against dense attention."""
    B, Hq, Hkv, C, M, page, T = 2, 4, 2, 128, 256, 32, 3
    g = torch.Generator().manual_seed(0)
    rot = xa.Rotary.make((64,))
    x = torch.randn(B, M, Hq + 2 * Hkv, C, generator=g).bfloat16().cuda()
    q, k, v = (t.transpose(1, 2) for t in x.split([Hq, Hkv, Hkv], 2))
    Q, K, V = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.arange(M, dtype=torch.int32, device="cuda")[:, None].contiguous()
    xa.xattn_rope(q, k, pos, rot, Q, K)
    tau = torch.full((Hq,), 1.0, device="cuda")
    bufs = xa.Buffers.allocate(B, Hq, M, C, 8, True, with_lse=True)
    O = xa.xattn_prefill(Q, K, V, tau, 8, True, bufs)

    c = xa.PagedCache.allocate(B, Hkv, C, 24, 12, page=page, eviction=True)
    for t in (c.k_pages, c.v_pages):
        t.fill_(float("nan"))
    c.lens.fill_(M)
    xa.xattn_cache_append(K, V, c)
    scale = 1 / math.sqrt(C)
    # the prompt's last token again, now through the cache: the prefill's own last row
    o, lse = run_decode(c, Q[:, :, -1], scale)
    check_decode(c, Q[:, :, -1], scale, o, lse)
    assert (f64(o) - f64(O[:, :, -1])).__abs__().max() < 2e-2      # the prefill's own bound
    # its log-sum-exp: the prefill exponentiates in part with a polynomial (1.1e-4)
    assert (lse - bufs.lse[:, :, -1]).abs().max() < 2e-4

    seen = c.lens.clone()
    ws = torch.empty(xa.xattn_decode_workspace_size(c, Hq, True), dtype=torch.uint8, device="cuda")
    budget = 200
    for step in range(2 * T):
        x = torch.randn(B, 1, Hq + 2 * Hkv, C, generator=g).bfloat16().cuda()
        q, k, v = (t.transpose(1, 2) for t in x.split([Hq, Hkv, Hkv], 2))
        c.lens += 1
        seen += 1
        qo, o, lse = (poisoned((B, Hq, 1, C), torch.bfloat16), poisoned((B, Hq, 1, C), torch.bfloat16),
                      poisoned((B, Hq)))
        xa.xattn_rope_append(q, k, v, (seen - 1).view(B, 1, 1), rot, c, qo, seen=seen)
        before = f64(c.acc)
        xa.xattn_decode_attn(qo, c, scale, o, ws, lse=lse, weights=True)
        check_decode(c, qo[:, :, 0], scale, o[:, :, 0], lse, before, f64(c.acc))
        if step == T - 1:
            want = do.cache_evict(to_oracle(c), budget, 16, 4, seen.cpu().numpy())
            run_evict(c, budget, 16, 4, seen)
            c.lens.clamp_(max=budget)
            np.testing.assert_array_equal(f64(c.k_pages), want["k"])
            np.testing.assert_array_equal(c.ordinal.cpu().numpy(), want["ordinal"])
            for b in range(B):      # the safe tokens are all still there
                for h in range(Hkv):
                    left = set(int(t) for t in do.cache_rows(to_oracle(c), "ordinal", b, h))
                    assert set(range(M + T - 16, M + T)) | set(range(4)) <= left


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_step_is_its_two_calls(e4m3):
    B, Hq, Hkv, C = 3, 8, 2, 64
    a = make_cache(6, [40, 1, 16], Hkv, C, 16, e4m3)
    b = clone_cache(a)
    x = torch.randn(B, 1, Hq + 2 * Hkv, C, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    q, k, v = (t.transpose(1, 2) for t in x.split([Hq, Hkv, Hkv], 2))
    rot, pos = xa.Rotary.make((32,)), (a.lens - 1).view(B, 1, 1)
    bufs = xa.DecodeBuffers.allocate(a, Hq, weights=True, with_lse=True)
    for t in (bufs.Q, bufs.O, bufs.lse, bufs.workspace):
        t.view(torch.uint8).fill_(0xFF)
    o = xa.xattn_decode_step(q, k, v, pos, rot, a, bufs, weights=True)
    qo = poisoned((B, Hq, 1, C), torch.bfloat16)
    xa.xattn_rope_append(q, k, v, pos, rot, b, qo)
    before = f64(b.acc)
    o2, lse2 = run_decode(b, qo[:, :, 0], 0.125, True)
    assert torch.equal(o[:, :, 0], o2) and torch.equal(bufs.lse, lse2) and same_cache(a, b)
    check_decode(b, qo[:, :, 0], 0.125, o2, lse2, before, f64(b.acc))


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_step_with_idle_sequences(e4m3):
    """A batch in which one sequence is empty, one has finished and one waits: the others' step
    is that of a batch without them, and theirs writes nothing but zero outputs."""
    Hq, Hkv, C, lens = 8, 2, 64, [40, 0, 33, 1, 200]
    c = make_cache(61, lens, Hkv, C, 16, e4m3)
    go = torch.tensor([1, 0, 0, 1, 0], dtype=torch.int32, device="cuda")
    on = [0, 3]
    x = torch.randn(5, 1, Hq + 2 * Hkv, C, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    x[~go.bool()] = float("nan")                       # an idle row holds anything
    q, k, v = (t.transpose(1, 2) for t in x.split([Hq, Hkv, Hkv], 2))
    rot, seen = xa.Rotary.make((32,)), c.lens + 7
    pos = (seen - 1).view(5, 1, 1)
    want = clone_cache(c)
    few = xa.PagedCache(want.k_pages, want.v_pages, want.page_table[on].contiguous(), want.lens[on].contiguous(),
                        want.k_scale, want.v_scale, want.acc, want.ordinal)
    fbufs = xa.DecodeBuffers.allocate(few, Hq, weights=True, with_lse=True)
    xa.xattn_decode_step(q[on], k[on], v[on], pos[on].contiguous(), rot, few, fbufs, seen=seen[on].contiguous(),
                         weights=True)
    bufs = xa.DecodeBuffers.allocate(c, Hq, weights=True, with_lse=True)
    for t in (bufs.Q, bufs.O, bufs.lse, bufs.workspace):
        t.view(torch.uint8).fill_(0xFF)
    o = xa.xattn_decode_step(q, k, v, pos, rot, c, bufs, seen=seen, weights=True, n_new=go)
    assert same_cache(c, want)
    assert torch.equal(o[~go.bool()], torch.zeros_like(o[~go.bool()]))
    assert torch.isneginf(bufs.lse[~go.bool()]).all()
    # (an idle sequence has no tiles, so the work is split as without it: the same bits)
    assert torch.equal(o[on], fbufs.O) and torch.equal(bufs.lse[on], fbufs.lse)
    assert _error() == xa.XATTN_OK
    # nobody has a token; then counts that are none
    before = clone_cache(c)
    for n, want_error in ((0, xa.XATTN_OK), (2, xa.XATTN_EINVAL), (-1, xa.XATTN_EINVAL), (2 ** 31 - 1, xa.XATTN_EINVAL)):
        o = xa.xattn_decode_step(q, k, v, pos, rot, c, bufs, seen=seen, weights=True, n_new=torch.full_like(go, n))
        assert _error() == want_error
        assert (o == 0).all() and torch.isneginf(bufs.lse).all() and same_cache(c, before)


def test_captured_step_with_changing_idle_sequences():
    """One capture of a step serves every later batch: which sequences are idle is read on the device."""
    Hq, Hkv, C, B = 4, 2, 64, 3
    start = make_cache(62, [40, 7, 200], Hkv, C, 16)
    c = clone_cache(start)
    x = torch.randn(B, 1, Hq + 2 * Hkv, C, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    q, k, v = (t.transpose(1, 2) for t in x.split([Hq, Hkv, Hkv], 2))
    rot, pos, go = xa.Rotary.make((32,)), (c.lens - 1).view(B, 1, 1), torch.ones(B, dtype=torch.int32, device="cuda")
    bufs = xa.DecodeBuffers.allocate(c, Hq, weights=True, with_lse=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        xa.xattn_decode_step(q, k, v, pos, rot, c, bufs, weights=True, n_new=go)
    for which in ([1, 1, 1], [0, 1, 0], [0, 0, 0], [1, 0, 1]):
        go.copy_(torch.tensor(which))
        for a, b in ((c.k_pages, start.k_pages), (c.v_pages, start.v_pages), (c.acc, start.acc),
                     (c.ordinal, start.ordinal)):
            a.copy_(b)
        bufs.O.fill_(float("nan"))
        g.replay()
        want, wbufs = clone_cache(start), xa.DecodeBuffers.allocate(c, Hq, weights=True, with_lse=True)
        xa.xattn_decode_step(q, k, v, pos, rot, want, wbufs, weights=True, n_new=go.clone())
        assert torch.equal(bufs.O, wbufs.O) and torch.equal(bufs.lse, wbufs.lse) and same_cache(c, want)
        for b in range(B):
            assert (bufs.O[b] == 0).all() == (not which[b])


def test_on_a_side_stream_and_in_graphs():
    """A decoding step captured into a graph and replayed with new inputs, lengths and pages,
    next to another graph with a workspace of its own."""
    B, Hq, Hkv, C, page = 2, 8, 2, 64, 16
    rot = xa.Rotary.make((32,))
    scale = 0.125

    def setup(seed):
        c = make_cache(seed, [40, 21], Hkv, C, page, slack=1)
        q = torch.randn(B, Hq, 1, C, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
        kv = torch.randn(2, B, Hkv, 1, C, generator=torch.Generator().manual_seed(seed + 9)).bfloat16().cuda()
        seen = c.lens.clone()
        pos = (seen - 1).view(B, 1, 1).clone()
        bufs = dict(qo=torch.empty_like(q), o=torch.empty_like(q), lse=torch.empty(B, Hq, device="cuda"),
                    ws=torch.empty(xa.xattn_decode_workspace_size(c, Hq, True), dtype=torch.uint8, device="cuda"),
                    ews=torch.empty(xa.xattn_cache_evict_workspace_size(c, 30), dtype=torch.uint8, device="cuda"))
        return c, q, kv, seen, pos, bufs

    def step(c, q, kv, seen, pos, m):
        xa.xattn_rope_append(q, kv[0], kv[1], pos, rot, c, m["qo"], seen=seen)
        xa.xattn_decode_attn(m["qo"], c, scale, m["o"], m["ws"], lse=m["lse"], weights=True)
        xa.xattn_cache_evict(c, 30, m["ews"], recent=4, seen=seen)

    sets, graphs = [setup(1), setup(2)], []
    step(*sets[0])                                    # first call outside any capture
    sets = [setup(1), setup(2)]
    for s in sets:
        gph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gph):
            step(*s)
        graphs.append(gph)
    sets_now = [setup(11), setup(12)]
    for s, new in zip(sets, sets_now):                # other inputs into the captured tensors
        for a, b in zip((s[0].k_pages, s[0].v_pages, s[0].page_table, s[0].lens, s[0].acc, s[0].ordinal, s[1],
                         s[2], s[3], s[4]),
                        (new[0].k_pages, new[0].v_pages, new[0].page_table, new[0].lens, new[0].acc,
                         new[0].ordinal, new[1], new[2], new[3], new[4])):
            a.copy_(b)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for gph, st in zip(graphs, side):
        with torch.cuda.stream(st):
            gph.replay()
    torch.cuda.synchronize()
    for s, new in zip(sets, sets_now):
        st = torch.cuda.Stream()
        xa.xattn_rope_append(new[1], new[2][0], new[2][1], new[4], rot, new[0], new[5]["qo"], seen=new[3],
                             stream=st)
        xa.xattn_decode_attn(new[5]["qo"], new[0], scale, new[5]["o"], new[5]["ws"], lse=new[5]["lse"],
                             weights=True, stream=st)
        xa.xattn_cache_evict(new[0], 30, new[5]["ews"], recent=4, seen=new[3], stream=st)
        torch.cuda.synchronize()
        assert torch.equal(s[5]["o"], new[5]["o"]) and torch.equal(s[5]["lse"], new[5]["lse"])
        assert same_cache(s[0], new[0])


def test_captured_step_after_a_fork():
    """In a capture, calls behind a join of two streams and behind a copy, whose predecessors are
    not just one kernel."""
    c = make_cache(54, [40, 21], 2, 64, 16)
    q = torch.randn(2, 8, 1, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    kv = torch.randn(2, 2, 2, 1, 64, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    src = [c.lens.clone(), c.page_table.clone()]
    rot, pos = xa.Rotary.make((32,)), (c.lens - 1).view(2, 1, 1).clone()
    qo, o = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(xa.xattn_decode_workspace_size(c, 8, True), dtype=torch.uint8, device="cuda")
    ref = clone_cache(c)
    xa.xattn_rope_append(q, kv[0], kv[1], pos, rot, ref, qo)
    xa.xattn_decode_attn(qo, ref, 0.125, o, ws, weights=True)
    want = o.clone()
    c.lens.zero_()
    c.page_table.fill_(-1)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            c.lens.copy_(src[0])
        c.page_table.copy_(src[1])
        main.wait_stream(side)
        xa.xattn_rope_append(q, kv[0], kv[1], pos, rot, c, qo)
        xa.xattn_decode_attn(qo, c, 0.125, o, ws, weights=True)
        c.lens.add_(0)
    o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and same_cache(c, ref)


def test_steps_without_a_pause_equal_steps_with_one():
    """Lengths, pages and queries change between calls that nothing waits for; the same steps
    with a synchronisation after every call give the same bits. (The calls overlap their
    set-up with the work ahead of them; what they read must not be from before it.)"""
    B, Hq, Hkv, C, page, steps = 3, 8, 2, 64, 16, 40
    rot = xa.Rotary.make((32,))
    g = torch.Generator().manual_seed(4)
    xs = torch.randn(steps, B, 1, Hq + 2 * Hkv, C, generator=g).bfloat16().cuda()
    start = make_cache(8, [40, 3, 0], Hkv, C, page, slack=3, spare=40)
    free = [p for p in range(start.num_pages) if p not in set(start.page_table.flatten().tolist())]
    fresh = torch.tensor(free, dtype=torch.int32).cuda()

    def go(pause):
        c = clone_cache(start)
        seen, taken, out = c.lens.clone(), 0, []
        ws = torch.empty(xa.xattn_decode_workspace_size(c, Hq, True), dtype=torch.uint8, device="cuda")
        ews = torch.empty(xa.xattn_cache_evict_workspace_size(c, 44), dtype=torch.uint8, device="cuda")
        lens = [40, 3, 0]
        for i in range(steps):
            for b in range(B):
                if lens[b] % page == 0 and lens[b] // page >= -(-[40, 3, 0][b] // page) \
                        and int(start.page_table[b, lens[b] // page]) < 0:
                    c.page_table[b, lens[b] // page].copy_(fresh[taken])
                    taken += 1
                lens[b] += 1
            c.lens.add_(1)
            seen.add_(1)
            q, k, v = (t.transpose(1, 2) for t in xs[i].split([Hq, Hkv, Hkv], 2))
            qo, o, lse = torch.empty_like(q.contiguous()), torch.empty(B, Hq, 1, C, dtype=torch.bfloat16,
                                                                       device="cuda"), torch.empty(B, Hq, device="cuda")
            for call in (lambda: xa.xattn_rope_append(q, k, v, (seen - 1).view(B, 1, 1), rot, c, qo, seen=seen),
                         lambda: xa.xattn_decode_attn(qo, c, 0.125, o, ws, lse=lse, weights=True),
                         lambda: xa.xattn_cache_evict(c, 44, ews, recent=8, seen=seen)):
                call()
                if pause:
                    torch.cuda.synchronize()
            c.lens.clamp_(max=44)
            lens = [min(n, 44) for n in lens]
            out += [o.clone(), lse.clone()]
        return c, out

    (a, oa), (b, ob) = go(False), go(True)
    assert all(torch.equal(x, y) for x, y in zip(oa, ob))
    assert same_cache(a, b) and torch.equal(a.lens, b.lens)
    assert not any(torch.isnan(x).any() for x in oa)


def test_pool_beyond_32_bit_offsets():
    """Pages whose element offsets pass 2^31 (and byte offsets 2^32): append, decode and
    evict there give what they give in a small pool."""
    Hkv, page, C, n = 8, 128, 128, 300
    P = 2 ** 31 // (Hkv * page * C) + 8
    small = make_cache(3, [n], Hkv, C, page)
    fill_eviction(small, 1)
    big = xa.PagedCache.allocate(1, Hkv, C, P, small.max_pages, page=page, eviction=True)
    ids = torch.tensor([P - 1, P - 4, P - 2], dtype=torch.int32).cuda()
    big.page_table[0, :3] = ids
    big.lens.copy_(small.lens)
    for a, b in ((big.k_pages, small.k_pages), (big.v_pages, small.v_pages), (big.acc, small.acc),
                 (big.ordinal, small.ordinal)):
        a[ids.long()] = b[small.page_table[0, :3].long()]
    g = torch.Generator().manual_seed(0)
    kv = torch.randn(2, 1, Hkv, 5, C, generator=g).bfloat16().cuda()
    q = torch.randn(1, 16, C, generator=g).bfloat16().cuda()
    out = []
    for c in (small, big):
        xa.xattn_cache_append(kv[0], kv[1], c)
        o, lse = run_decode(c, q, 0.1, True)
        run_evict(c, 100, 10, 2)
        pg = c.page_table[0, :3].long()
        out.append([o, lse] + [raw(t[pg]) for t in (c.k_pages, c.v_pages, c.acc, c.ordinal)])
    for a, b in zip(*out):
        assert torch.equal(a, b)


# --------------------------------------- what only the device can see, as an error word
def _error():
    return xa.xattn_get_device_error()


@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
def test_bad_pages_touch_nothing_and_raise(bad):
    C = 64
    c = make_cache(2, [40, 50], 2, C, 16)
    fill_eviction(c, 1)
    c.page_table[0, 1] = bad                          # slots 16..31 of sequence 0
    q = torch.randn(2, 4, C, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    assert _error() == xa.XATTN_OK
    before = clone_cache(c)
    o, lse = run_decode(c, q, 0.1, True)
    assert _error() == xa.XATTN_EINVAL and _error() == xa.XATTN_OK
    # the other sequence is not affected
    fine = clone_cache(before)
    fine.page_table[0, 1] = fine.page_table[0, 0]
    o2, lse2 = run_decode(fine, q, 0.1)
    assert _error() == xa.XATTN_OK
    assert torch.equal(o[1], o2[1]) and torch.equal(lse[1], lse2[1])
    kv = torch.randn(2, 2, 2, 12, C, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    c = clone_cache(before)
    xa.xattn_cache_append(kv[0], kv[1], c)            # slots 28..39 of sequence 0
    assert _error() == xa.XATTN_EINVAL
    assert torch.equal(c.k_pages[before.page_table[0, 2].long(), :, :8], kv[0][0, :, 4:])
    ws = poisoned(xa.xattn_cache_evict_workspace_size(c, 20), torch.uint8)
    xa.xattn_cache_evict(c, 20, ws, recent=2)
    assert _error() == xa.XATTN_EINVAL


def test_append_beside_a_bad_page_writes_its_own_slots_only():
    """Every pool row after an append that reaches a bad page."""
    c = make_cache(53, [40, 50], 2, 64, 16)
    fill_eviction(c, 1)
    c.page_table[0, 1] = -1                       # slots 16..31 of sequence 0
    before = clone_cache(c)
    kv = torch.randn(2, 2, 2, 20, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    xa.xattn_cache_append(kv[0], kv[1], c)        # slots 20..39 and 30..49
    assert _error() == xa.XATTN_EINVAL
    want = clone_cache(before)
    for b, n in ((0, 40), (1, 50)):
        for s in range(n - 20, n):
            pg, r = int(before.page_table[b, s // 16]), s % 16
            if pg < 0:
                continue
            want.k_pages[pg, :, r], want.v_pages[pg, :, r] = kv[0][b, :, s - n + 20], kv[1][b, :, s - n + 20]
            want.acc[pg, :, r], want.ordinal[pg, :, r] = 0, s
    assert same_cache(c, want)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens,Hkv,page,budget,bad", [
    ([100, 57], 2, 16, 50, [1]),               # below the budget
    ([100, 57], 2, 16, 50, [4]),               # above it
    ([100, 57], 2, 16, 50, [3]),               # across it
    ([100, 57], 1, 16, 50, [0, 1, 2, 3, 4]),
    ([100, 57], 1, 16, 50, [0, 1, 2, 3, 4, 5, 6]),   # every page
    ([9000, 100], 1, 64, 4000, [0, 7, 62, 63, 100, 140]),      # a cluster of CTAs
])
def test_evict_leaves_bad_pages_out(lens, Hkv, page, budget, bad, e4m3):
    """Slots of bad pages keep their places below the budget; of the others as many stay as have
    a place there, and none of them is lost. Nothing else is written."""
    c = make_cache(51, lens, Hkv, 64, page, e4m3)
    fill_eviction(c, 3, ties=True)
    good = c.page_table.clone()
    c.page_table[0, bad] = torch.tensor([-1, c.num_pages, 2 ** 31 - 1], dtype=torch.int32).cuda()[
        torch.arange(len(bad)) % 3]
    before, seen = to_oracle(c), (3 * c.lens).cpu().numpy()
    want = do.cache_evict(dict(before, lens=np.array([0, lens[1]]), table=good.cpu().numpy()), budget, 8, 4, seen)
    where = {s: do.cache_slot(before, 0, s) for s in range(lens[0]) if s // page not in bad}
    n = min(budget, lens[0])
    room = sum(s < n for s in where)
    for h in range(Hkv):
        slots = sorted(where)
        kept = do.evict_kept([before["acc"][where[s][0], h, where[s][1]] for s in slots],
                             [before["ordinal"][where[s][0], h, where[s][1]] for s in slots], room, seen[0], 8, 4)
        kept = {slots[i] for i in kept}
        holes = [s for s in slots if s < n and s not in kept]
        movers = sorted((s for s in kept if s >= n), reverse=True)
        assert len(holes) == len(movers)
        for to, frm in zip(holes, movers):
            for name in ("k", "v", "acc", "ordinal"):
                want[name][where[to][0], h, where[to][1]] = before[name][where[frm][0], h, where[frm][1]]
    assert _error() == xa.XATTN_OK
    acc_out, ord_out = c.acc.clone(), c.ordinal.clone()
    apart = clone_cache(c)
    run_evict(apart, budget, 8, 4, 3 * c.lens, acc_out=acc_out, ord_out=ord_out)
    assert _error() == xa.XATTN_EINVAL
    run_evict(c, budget, 8, 4, 3 * c.lens)
    assert _error() == xa.XATTN_EINVAL
    for name, x, y in (("k", c.k_pages, apart.k_pages), ("v", c.v_pages, apart.v_pages), ("acc", c.acc, acc_out),
                       ("ordinal", c.ordinal, ord_out)):
        np.testing.assert_array_equal(f64(x), want[name])
        assert torch.equal(raw(x), raw(y))


def test_bad_lengths_and_counts_touch_nothing_and_raise():
    C = 64
    c = make_cache(2, [40, 50], 2, C, 16)
    cap = c.max_pages * c.page
    before = clone_cache(c)
    q = torch.randn(2, 4, C, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    good, _ = run_decode(c, q, 0.1)
    for n in (-1, cap + 1, 2 ** 31 - 1, -2 ** 31):
        c.lens[0] = n
        o, lse = run_decode(c, q, 0.1)
        assert _error() == xa.XATTN_EINVAL
        assert (o[0] == 0).all() and torch.isneginf(lse[0]).all() and torch.equal(o[1], good[1])
        c2 = clone_cache(c)
        c2.lens[1] = 5                                # below the budget: nothing may move
        ws = poisoned(xa.xattn_cache_evict_workspace_size(c, 20), torch.uint8)
        xa.xattn_cache_evict(c2, 20, ws, recent=2)
        assert _error() == xa.XATTN_EINVAL
        assert same_cache(c2, c)
        kv = torch.zeros(2, 2, 2, 3, C).bfloat16().cuda()
        c2 = clone_cache(c)
        xa.xattn_cache_append(kv[0], kv[1], c2, n_new=torch.tensor([3, 0], dtype=torch.int32).cuda())
        assert _error() == xa.XATTN_EINVAL
        assert same_cache(c2, c)
    c = clone_cache(before)
    kv = torch.ones(2, 2, 2, 3, C).bfloat16().cuda()
    for new in ([-1, 0], [4, 0]):                     # outside [0, T]
        c2 = clone_cache(c)
        xa.xattn_cache_append(kv[0], kv[1], c2, n_new=torch.tensor(new, dtype=torch.int32).cuda())
        assert _error() == xa.XATTN_EINVAL
        assert same_cache(c2, c)
    c.lens[0] = 2                                     # more new tokens than slots
    c2 = clone_cache(c)
    xa.xattn_cache_append(kv[0], kv[1], c2, n_new=torch.tensor([3, 0], dtype=torch.int32).cuda())
    assert _error() == xa.XATTN_EINVAL
    assert same_cache(c2, c)


def test_binding_refuses_on_the_gpu_too():
    c = make_cache(2, [40, 50], 2, 64, 16, eviction=False)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(xa.xattn_decode_workspace_size(c, 4), dtype=torch.uint8, device="cuda")
    o = torch.empty_like(q)
    with pytest.raises(ValueError, match="acc"):
        xa.xattn_decode_attn(q, c, 0.1, o, ws, weights=True)
    with pytest.raises(ValueError, match="acc_out"):
        xa.xattn_decode_attn(q, c, 0.1, o, ws, acc_out=torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        xa.xattn_decode_attn(q[:1], c, 0.1, o[:1], ws)
    with pytest.raises(xa.XAttnError):
        xa.xattn_decode_attn(q[:, :3], c, 0.1, o[:, :3].contiguous(), ws)
    with pytest.raises(xa.XAttnError):
        xa.xattn_decode_attn(q, c, 0.1, o, ws[:128])
    with pytest.raises(ValueError, match="acc and ordinal"):
        xa.xattn_cache_evict(c, 10, ws)
    with pytest.raises(ValueError, match="CUDA"):
        xa.xattn_decode_attn(q, c, 0.1, o, ws.cpu())
    with pytest.raises(AttributeError):
        c.lens = c.lens.clone()
    c = make_cache(2, [40, 50], 2, 64, 16)
    for kw in (dict(budget=2 ** 32 + 5), dict(budget=-1), dict(budget=10, recent=2 ** 32), dict(budget=10, sink=-1)):
        with pytest.raises(ValueError, match="count"):
            xa.xattn_cache_evict(c, workspace=ws, **kw)
    with pytest.raises(xa.XAttnError):
        xa.xattn_cache_evict(c, 0, ws)
